/*
 * gdn.h -- C ABI of the Gated DeltaNet (GDN) layer core forward on GB300 (sm_103a).
 *
 * The core forward computes, per token t and v head h (GQA: v head h reads q/k
 * head h / (Hv/Hk)):
 *
 *   1. a width-4 causal depthwise convolution over the channel-concatenated
 *      [q_raw | k_raw | v_raw] projections followed by SiLU
 *      ("fused q/k/v short conv", flash-linear-attention PR #972, sections
 *      "Summary" and "Why"; "GDN Elementwise Fusion", option table, pre-GDR);
 *   2. per-head L2 normalisation of q and k, x * rsqrt(sum x^2 + 1e-6)
 *      ("perf(gated_delta_net): fold q/k L2-norm into the gated_delta_rule
 *      kernel", Megatron-LM PR #5396, section "Why");
 *   3. beta = sigmoid(b) and the decay g = -exp(A_log) * softplus(a + dt_bias)
 *      ("GDN Elementwise Fusion", option table: beta and decay preparation);
 *   4. the gated delta rule S_t = exp(g_t) S_{t-1} (I - beta_t k_t k_t^T)
 *      + beta_t v_t k_t^T, o_t = scale * S_t q_t, evaluated chunk by chunk
 *      (64 tokens, WY/UT form) with an fp32 state;
 *   5. y = RMSNorm(o) * SiLU(gate), the RMSNorm result materialised in the
 *      activation dtype before the fp32 gating multiply ("GDN Elementwise
 *      Fusion", post-GDR requirements and "Execution and numerical behavior").
 *
 * Conventions shared by every entry point:
 *  - All tensor pointers are DEVICE pointers owned by the caller. The library
 *    never allocates, frees or synchronises (except gdn_device_status, which
 *    says so). Every call is asynchronous on `stream` (0 = legacy default).
 *  - Return value: GDN_OK (0) or a negative gdn_status. Argument checks read
 *    metadata only (no device synchronisation). On an error nothing is
 *    launched. There is no fallback path for unsupported inputs.
 *  - Element strides are in elements of the tensor's own dtype; the channel
 *    (last) dimension is always contiguous.
 *  - Device-side argument faults (a malformed cu_seqlens) cannot be seen by
 *    the host without a sync: the kernels then write a status word in the
 *    workspace and skip their work; read it with gdn_device_status().
 */
#ifndef GDN_H
#define GDN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st *gdn_stream_t; /* == cudaStream_t */

typedef enum {
    GDN_OK = 0,
    GDN_ERR_INVALID_ARG = -1,  /* null pointer, non-positive size, bad stride or alignment */
    GDN_ERR_UNSUPPORTED = -2,  /* dk/dv not a power of two in [16, 512], conv_width != 4,
                                  Hv % Hk != 0, unsupported dtype combination */
    GDN_ERR_WORKSPACE = -3,    /* workspace missing, misaligned or smaller than
                                  gdn_workspace_bytes() */
    GDN_ERR_CUDA = -4,         /* a CUDA launch or query failed */
    GDN_ERR_DEVICE_SEQLENS = -5, /* (device status) cu_seqlens not 0-based, not
                                    non-decreasing or not ending at T */
    GDN_ERR_DEVICE_RANGE = -6,  /* (device status) a non-finite gated-delta-rule output
                                   reached step 5 (the separate output kernel, or the
                                   output step inside the chunk kernel): a non-finite
                                   input, or a value beyond the fp16 range of the
                                   intermediates */
    GDN_ERR_DEVICE_TIMEOUT = -7 /* (device status) a tensor-core kernel gave up waiting
                                   (about 1 s) for a copy or an MMA; results are invalid */
} gdn_status;

typedef enum { GDN_F32 = 0, GDN_BF16 = 1, GDN_F16 = 2 } gdn_dtype;

/* Problem descriptor. Fill it with gdn_desc_init() and then override
 * strides/dtypes of views as needed. */
typedef struct {
    int32_t B, T;        /* batch rows, tokens per row; with cu_seqlens: B = 1 and
                            T = total packed tokens */
    int32_t N;           /* sequences: B without cu_seqlens, else cu_seqlens has N+1 entries */
    int32_t Hk, Hv;      /* q/k heads, v heads (Hv % Hk == 0) */
    int32_t dk, dv;      /* head dims: powers of two in [16, 512] */
    int32_t conv_width;  /* short-conv taps; must be 4 */
    int32_t dtype;       /* gdn_dtype of q_raw, k_raw, v_raw, a, b, conv_w and out */
    int32_t gate_dtype;  /* dtype, or GDN_F32 */
    int32_t norm_w_dtype;/* dtype, or GDN_F32 */
    int32_t reserved0;
    /* (batch, token) element strides; channel stride is 1 */
    int64_t q_stride_b, q_stride_t;
    int64_t k_stride_b, k_stride_t;
    int64_t v_stride_b, v_stride_t;
    int64_t a_stride_b, a_stride_t;
    int64_t b_stride_b, b_stride_t;
    int64_t gate_stride_b, gate_stride_t;
    float l2_eps;        /* q/k L2-norm eps, 1e-6 */
    float norm_eps;      /* output RMSNorm eps, 1e-5 */
    float scale;         /* q scale in o_t = scale * S_t q_t, 1 */
    int32_t reserved1;
} gdn_desc;

/* Fill *d for contiguous tensors: q_raw/k_raw [B,T,Hk*dk], v_raw [B,T,Hv*dv],
 * a/b [B,T,Hv], gate [B,T,Hv*dv], gate/norm_w in the act dtype,
 * l2_eps 1e-6, norm_eps 1e-5, scale 1, conv_width 4. N = B when packed == 0;
 * packed != 0 requires B == 1 and sets N = packed. Returns the validation
 * status of the filled descriptor. */
int gdn_desc_init(gdn_desc *d, int B, int T, int packed, int Hk, int Hv, int dk, int dv,
                  int dtype);

/* Bytes of scratch the forward needs for *d (intermediate q/k/v, beta, the
 * in-chunk cumulative decay, o, a status word and the chunk table). */
int gdn_workspace_bytes(const gdn_desc *d, size_t *bytes);

/* Offsets (bytes from the workspace base) of the intermediate tensors, for
 * inspection by tests and tools:
 *   q, k [Hk][Ntok][dk] after conv, SiLU and L2 norm: fp32 for fp32
 *   activations, else two fp16 planes (hi = fp16(x) at the offset, then
 *   lo = fp16(x - hi) right after the Hk*Ntok*dk hi elements); v [Hv][Ntok][dv]
 *   after conv and SiLU and o [Ntok][Hv][dv] (gated delta rule output): fp16 for
 *   bf16/fp16 activations, fp32 for fp32 activations; beta [Hv][Ntok] fp32;
 *   gamma [Hv][Ntok] = in-chunk inclusive cumulative sum of g, fp64 for fp32
 *   activations and fp32 otherwise; status: int32 device status word;
 *   chunk_off: int32 [N+1]; tpt: the tensor-core kernels' region (empty where
 *   they do not run): per (v head, chunk slot) 32 KB of prep tiles (the 128x64
 *   fp16 tile [T; P T], then X), and for one sequence (N = 1) after them the fp32
 *   state handed between the segments of its chain, [Hv][dk][dv]. */
typedef struct {
    size_t status, chunk_off, q, k, v, beta, gamma, o, tpt, total;
} gdn_workspace_layout;
int gdn_workspace_offsets(const gdn_desc *d, gdn_workspace_layout *layout);

/*
 * The whole core forward (steps 1-5 above) on `stream`.
 *   q_raw, k_raw   act dtype, [B,T,Hk*dk] at (q|k)_stride_(b|t); 16-byte aligned
 *                  base and strides
 *   v_raw          act dtype, [B,T,Hv*dv] at v_stride_(b|t); 16-byte aligned
 *   a, b           act dtype, [B,T,Hv] at (a|b)_stride_(b|t); any alignment
 *   gate           gate_dtype, [B,T,Hv*dv] at gate_stride_(b|t): may be a strided,
 *                  unaligned view into a wider projection buffer
 *   conv_w         act dtype, [2*Hk*dk + Hv*dv][4] contiguous, q|k|v channel
 *                  order, tap 3 multiplies the current token; 16-byte aligned
 *   A_log, dt_bias fp32 [Hv]
 *   norm_w         norm_w_dtype [dv] contiguous
 *   cu_seqlens     NULL, or int32 [N+1] packed-sequence offsets (then B == 1);
 *                  the conv halo and the state restart at every offset
 *   initial_state  NULL (zeros) or fp32 [N][Hv][dk][dv], the transposed state
 *                  S^T of every (sequence, v head); 16-byte aligned
 *   out            act dtype [B,T,Hv,dv] contiguous; 16-byte aligned
 *                  (token tensors and out may be NULL when B*T == 0)
 *   final_state    NULL (not written) or fp32 [N][Hv][dk][dv]; 16-byte aligned
 *   workspace      device scratch of >= gdn_workspace_bytes(), 256-byte aligned;
 *                  calls that share a workspace must not overlap on the GPU
 * Inputs are only read; initial_state and final_state may alias.
 * Ordering: the call's first kernel starts after everything queued on `stream`
 * before it, and work queued after the call starts after its last kernel. On
 * the tensor-core path without segments the later kernels of the call are
 * programmatic dependents of the kernel before them (their CTAs may become
 * resident early and wait on the device); a long single sequence runs part of
 * the chunk stage on a high-priority stream the library creates once per
 * device, joined back to `stream` by events.
 */
int gdn_forward(const gdn_desc *d,
                const void *q_raw, const void *k_raw, const void *v_raw,
                const void *a, const void *b, const void *gate,
                const void *conv_w, const float *A_log, const float *dt_bias,
                const void *norm_w, const int32_t *cu_seqlens,
                const float *initial_state, void *out, float *final_state,
                void *workspace, size_t workspace_bytes, gdn_stream_t stream);

/* The three stages of gdn_forward, callable one by one on the same workspace
 * (gdn_forward gives bit for bit the results of prologue, chunk_rule, epilogue in
 * this order). Where the transposed tensor-core chunk kernel holds a whole v-head
 * row (16-bit activations, dk 64 or 128, dv = 128), the gate and norm_w match the
 * activation dtype (norm_w may be fp32), the gate view has a 16-byte aligned base
 * and row pitch with its batch rows back to back, and the chunk stage is not cut
 * into segments (one long sequence), gdn_forward applies step 5 inside that kernel,
 * with the same arithmetic, and leaves o in the workspace unwritten.
 * gdn_prologue: steps 1-3 plus the in-chunk cumulative decay -> workspace q, k,
 *   v, beta, gamma (and the chunk table / status word when cu_seqlens is set).
 * gdn_chunk_rule: step 4 -> workspace o, final_state.
 * gdn_epilogue: step 5 -> out. */
int gdn_prologue(const gdn_desc *d, const void *q_raw, const void *k_raw,
                 const void *v_raw, const void *a, const void *b, const void *conv_w,
                 const float *A_log, const float *dt_bias, const int32_t *cu_seqlens,
                 void *workspace, size_t workspace_bytes, gdn_stream_t stream);
int gdn_chunk_rule(const gdn_desc *d, const int32_t *cu_seqlens,
                   const float *initial_state, float *final_state,
                   void *workspace, size_t workspace_bytes, gdn_stream_t stream);
int gdn_epilogue(const gdn_desc *d, const void *gate, const void *norm_w, void *out,
                 void *workspace, size_t workspace_bytes, gdn_stream_t stream);

/* Wait for `stream`, then read the device status word of the last forward that
 * used `workspace` into *status (GDN_OK or a GDN_ERR_DEVICE_* code). This call
 * synchronises the stream. */
int gdn_device_status(const void *workspace, int *status, gdn_stream_t stream);

/* Static description of a status code. */
const char *gdn_status_string(int status);

/*
 * Test hook for the bounded waits (GDN_ERR_DEVICE_TIMEOUT) of the tensor-core kernels
 * and of the gated linear recurrence (below).
 * Every wait of those kernels on one of their own mbarriers gives up after about
 * a second; the CTA then records GDN_ERR_DEVICE_TIMEOUT, waits (again bounded) for
 * its own copies and products in flight, frees its tensor memory and returns.
 * With immediate = 1, calls made afterwards in this process launch these kernels
 * so that a main-loop wait which is not already complete gives up at once (a
 * non-blocking test instead of the timed wait), which drives that path on any
 * input without stalling the GPU; the drains keep their ~1 s limit. immediate = 0
 * restores the normal waits. The outputs of a call that timed out are
 * unspecified; the next call in the normal mode is unaffected. Not meant for
 * production use; there is no counterpart on the pages. Returns GDN_OK, or
 * GDN_ERR_INVALID_ARG for another value.
 */
int gdn_set_wait_test_mode(int immediate);

/*
 * gdn_forward without a caller-provided workspace, for callers that cannot
 * allocate device memory (code running inside another framework's memory
 * arena, plugins without an allocator, hosts that forbid allocation while
 * serving). The pages describe no such entry point; it has no counterpart there.
 *
 * The scratch is a fixed device array of GDN_STATIC_WORKSPACE_BYTES inside the
 * library; every GPU that loads the library holds it until the process exits.
 * Arguments and results are those of gdn_forward (same pointers, layouts and
 * status codes, without workspace and workspace_bytes).
 *  - Problems whose gdn_workspace_bytes() exceeds GDN_STATIC_WORKSPACE_BYTES are
 *    rejected with GDN_ERR_WORKSPACE before anything is launched.
 *  - The device is the current CUDA device; `stream` must belong to it. The
 *    first call on a device looks up the array's device address
 *    (cudaGetSymbolAddress); make that first call before any stream capture.
 *  - The call allocates nothing (no cudaMalloc, cudaFree or allocating library
 *    routine).
 *  - All calls on a device share the one array, which keeps the last call's
 *    contents: calls that overlap on the GPU (different streams, or host
 *    threads racing on one device) race on it and must be serialised by the
 *    caller.
 *  - Device-side status (GDN_ERR_DEVICE_SEQLENS, GDN_ERR_DEVICE_RANGE,
 *    GDN_ERR_DEVICE_TIMEOUT) goes to the status word at the start of the
 *    array, as gdn_forward's goes to its workspace; read it with
 *    gdn_static_ws_device_status below.
 *  - The address is looked up again when the device's context changes (e.g.
 *    after cudaDeviceReset), so a reset between calls is safe.
 */
#define GDN_STATIC_WORKSPACE_BYTES (16u * 1024u * 1024u)
int gdn_forward_static_ws(const gdn_desc *d,
                          const void *q_raw, const void *k_raw, const void *v_raw,
                          const void *a, const void *b, const void *gate,
                          const void *conv_w, const float *A_log, const float *dt_bias,
                          const void *norm_w, const int32_t *cu_seqlens,
                          const float *initial_state, void *out, float *final_state,
                          gdn_stream_t stream);

/* Wait for `stream`, then read the device status word of the last
 * gdn_forward_static_ws call on the current device into *status (GDN_OK or a
 * GDN_ERR_DEVICE_* code), like gdn_device_status for a caller's workspace. No
 * counterpart on the pages either. Synchronises the stream; allocates nothing.
 * Returns GDN_OK, GDN_ERR_INVALID_ARG (null status) or GDN_ERR_CUDA. */
int gdn_static_ws_device_status(int *status, gdn_stream_t stream);

/* Which gated-delta-rule kernel serves *d: 0 = fp32 CUDA-core kernel,
 * 1 = tcgen05 tensor-core kernel (bf16/fp16). */
int gdn_chunk_kernel_kind(const gdn_desc *d);

/*
 * Decode: one new token for each of d->B sequences. The result is what
 * gdn_forward gives for one more token of each sequence (same definitions,
 * same readings): the width-4 causal conv takes the sequence's last three raw
 * inputs from a conv cache, then SiLU, the q/k L2 norm, beta and the decay, one
 * step of S_t = exp(g_t) S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T with
 * o_t = scale * S_t q_t from the carried state, and the gated RMSNorm. The pages
 * define the forward; a decode cache appears there only as the conv input that a
 * fused prefill conv has to leave out ("fused q/k/v short conv",
 * flash-linear-attention PR #972, "Risk / scope").
 *
 * d           d->T == 1, not packed (N == B), everything else as for gdn_forward;
 *             the token tensors are [B, 1, *] views (only the batch strides and
 *             the contiguous channels matter).
 * q_raw ... norm_w   as for gdn_forward, one token per sequence.
 * conv_state  act dtype [B][ch][3] contiguous, ch = 2*Hk*dk + Hv*dv in q|k|v
 *             order: per channel the raw inputs of the sequence's last three
 *             tokens, oldest first (zeros where the sequence has fewer). Read,
 *             then overwritten with the window advanced by this token. After a
 *             gdn_forward prefill it holds that call's last three raw tokens.
 * state       fp32 [B][Hv][dk][dv] (S^T per sequence and v head, the layout of
 *             gdn_forward's initial_state / final_state), 16-byte aligned; read
 *             and overwritten in place.
 * out         act dtype [B, 1, Hv, dv] contiguous, 16-byte aligned.
 * workspace   gdn_decode_workspace_bytes(d) bytes, 256-byte aligned; its first
 *             word is the device status (gdn_device_status).
 * Returns GDN_OK or a negative status as gdn_forward (GDN_ERR_INVALID_ARG for
 * d->T != 1 or a packed descriptor). conv_state, state, out and workspace must
 * not overlap each other or the inputs.
 */
int gdn_decode_workspace_bytes(const gdn_desc *d, size_t *bytes);
int gdn_decode_step(const gdn_desc *d,
                    const void *q_raw, const void *k_raw, const void *v_raw,
                    const void *a, const void *b, const void *gate,
                    const void *conv_w, const float *A_log, const float *dt_bias,
                    const void *norm_w, void *conv_state, float *state, void *out,
                    void *workspace, size_t workspace_bytes, gdn_stream_t stream);

/*
 * gdn_forward for sequences that continue an earlier part (chunked prefill, or
 * one span of a sequence split across ranks): the width-4 causal conv reads the
 * raw inputs of the three tokens before each sequence from conv_prefix instead
 * of zeros ("fused q/k/v short conv", flash-linear-attention PR #972, "Summary":
 * a per-channel causal short conv over the projections; the earlier tokens are
 * the conv's left context). Everything else is gdn_forward's, with the state
 * carried in through initial_state.
 *
 * conv_prefix  act dtype [N][3][2*Hk*dk + Hv*dv] contiguous, 16-byte aligned:
 *              per sequence the raw q|k|v inputs (conv_w's channel order) of
 *              its three preceding tokens, oldest first; NULL = zeros (then
 *              this is gdn_forward).
 * Returns as gdn_forward (GDN_ERR_INVALID_ARG also for a misaligned prefix).
 */
int gdn_forward_with_prefix(const gdn_desc *d,
                            const void *q_raw, const void *k_raw, const void *v_raw,
                            const void *a, const void *b, const void *gate,
                            const void *conv_w, const float *A_log, const float *dt_bias,
                            const void *norm_w, const int32_t *cu_seqlens,
                            const void *conv_prefix, const float *initial_state,
                            void *out, float *final_state,
                            void *workspace, size_t workspace_bytes, gdn_stream_t stream);

/*
 * The exchange step of the sequence-sharded core. Over a span of one sequence
 * the chunked gated delta rule (S_t = exp(g_t) S_{t-1} (I - beta_t k_t k_t^T) +
 * beta_t v_t k_t^T, state H = S^T) is affine in the span's initial state:
 * H_end = A H_start + B, where B is the span's final state from zeros and A
 * (dk x dk) the span's final state with v = 0, dv = dk and the identity as
 * initial state (both by gdn_forward_with_prefix). Given every span's maps in
 * sequence order, this writes each span's initial state:
 *     H_in[0] = h0,  H_in[s] = A[s-1] H_in[s-1] + B[s-1].
 *
 * spans      number of spans (0: nothing to do).
 * A          fp32 [spans][Hv][dk][dk]; B fp32 [spans][Hv][dk][dv] (the last
 *            span's maps are not read); h0 fp32 [Hv][dk][dv] or NULL (zeros);
 * H_in       fp32 [spans][Hv][dk][dv], written.
 * All device pointers, 16-byte aligned. Returns GDN_OK, GDN_ERR_INVALID_ARG
 * (bad size, null or misaligned pointer) or GDN_ERR_CUDA. Asynchronous on
 * stream; H_in must not overlap A, B or h0.
 */
int gdn_span_scan(int spans, int Hv, int dk, int dv, const float *A, const float *B,
                  const float *h0, float *H_in, gdn_stream_t stream);

/*
 * Backward of the core: the gradients of
 *     L = sum(grad_out * out) + sum(grad_final * final_state)
 * with respect to every input of gdn_forward, first order. The pages define
 * the forward; training needs its first-order gradients ("GDN Elementwise
 * Fusion", Megatron Core developer guide, "Execution and numerical behavior":
 * the fused post-GDR kernels support first-order autograd; "fused q/k/v short
 * conv", flash-linear-attention PR #972, "Test plan": input and parameter
 * gradients of the fused path checked against the unfused one, and the
 * benchmark table timing forward + backward). Reading: the rounding of the
 * RMSNorm result to the activation dtype is taken as the identity (the
 * straight-through derivative of the rounded forward).
 *
 * The call recomputes the forward, storing each chunk's start state, and then
 * runs the reverse pass. What runs depends on the activation dtype:
 *  - fp32 activations: everything on CUDA cores in fp32 (the prologue, a
 *    state recompute, the reverse pass);
 *  - 2-byte activations with dk in {64, 128, 256} and dv a multiple of 64
 *    (gdn_chunk_kernel_kind() == 1): the forward's tcgen05 chunk stage (prep
 *    and chain) recomputes the states, the new values and the outputs in fp32;
 *    the dO' terms and the per-chunk dv contractions are tcgen05 products
 *    (split bf16 or fp16 operands, fp32 accumulators);
 *  - other 2-byte shapes: an fp32 CUDA-core state recompute; where dk and dv
 *    are multiples of 64 (dv <= 512) the outputs and the dO' terms are still
 *    tcgen05 products;
 *  - in every case the serial reverse chain, the per-chunk gradients' other
 *    terms and the elementwise backward run on CUDA cores in fp32.
 * Every sum has a fixed order: results are run-to-run identical.
 *
 * d, q_raw ... initial_state   exactly as for gdn_forward (same descriptor,
 *             strides, packing and alignment rules).
 * grad_out    act dtype [B*T][Hv][dv] contiguous (the gradient of out).
 * grad_final  fp32 [N][Hv][dk][dv] (S^T layout of final_state), or NULL = zeros.
 * dq_raw, dk_raw  act dtype, dense [B*T][Hk*dk]; dv_raw act dtype [B*T][Hv*dv];
 *             these three 16-byte aligned;
 * da, db      act dtype [B*T][Hv]; dgate gate dtype [B*T][Hv*dv] (all dense,
 *             whatever the strides of the inputs);
 * dconv_w     fp32 [2*Hk*dk+Hv*dv][4]; dA_log, ddt_bias fp32 [Hv];
 * dnorm_w     fp32 [dv]; dinitial_state fp32 [N][Hv][dk][dv] or NULL (skip).
 *             All outputs are written in full (not accumulated into).
 * workspace   gdn_backward_workspace_bytes(d) bytes, 256-byte aligned; it
 *             begins with gdn_forward's layout (status word first, so
 *             gdn_device_status reads it), followed by the backward's fp32
 *             regions: per token and v head about 2*dk*dv/64 + 3*dv + 2*dk + 196
 *             floats, plus 2*Hk*dk + Hv*dv floats per token (about 180 KB per
 *             token at 6 heads, dk 256, dv 512).
 * Returns GDN_OK, GDN_ERR_INVALID_ARG (null or misaligned pointer),
 * GDN_ERR_UNSUPPORTED (as gdn_forward), GDN_ERR_WORKSPACE or GDN_ERR_CUDA; a
 * malformed cu_seqlens sets GDN_ERR_DEVICE_SEQLENS in the workspace and the
 * kernels skip their work. Outputs must not overlap the inputs or workspace.
 */
int gdn_backward_workspace_bytes(const gdn_desc *d, size_t *bytes);
int gdn_backward(const gdn_desc *d,
                 const void *q_raw, const void *k_raw, const void *v_raw,
                 const void *a, const void *b, const void *gate,
                 const void *conv_w, const float *A_log, const float *dt_bias,
                 const void *norm_w, const int32_t *cu_seqlens,
                 const float *initial_state, const void *grad_out,
                 const float *grad_final, void *dq_raw, void *dk_raw, void *dv_raw,
                 void *da, void *db, void *dgate, float *dconv_w, float *dA_log,
                 float *ddt_bias, float *dnorm_w, float *dinitial_state,
                 void *workspace, size_t workspace_bytes, gdn_stream_t stream);

/*
 * ---------------------------------------------------------------------------
 * Operators of the layers that stand beside the gated delta rule: a gated
 * linear recurrence with one state value per channel, rotary positions, and
 * group norm with an activation. They follow the conventions at the top of this
 * file (device pointers, no allocation, no synchronisation, metadata checks
 * only, a status word in the workspace where the device checks something). The
 * pages describe none of them; their definitions stand here in full.
 *
 * Alignment: every tensor needs the alignment of its own element type; rows that
 * are 16-byte aligned (base pointer, strides and row length) take the vector
 * kernels, others element-wise ones. The two agree to the rounding of fp32
 * arithmetic (the recurrence and the group norm add up in another order).
 * "Run-to-run identical" below means calls of the same sizes and alignment.
 */

/*
 * Gated linear recurrence. Per sequence and channel c, with the decay written as
 * the gated delta rule's:
 *     g_t     = -exp(A_log[c]) * softplus(a_t + dt_bias[c])      (<= 0)
 *     alpha_t = exp(g_t)
 *     u_t     = sqrt(1 - alpha_t^2) * sigmoid(b_t) * x_t
 *     h_t     = alpha_t * h_{t-1} + u_t,        out_t = h_t
 * h before a sequence's first token is its initial state (zeros without one).
 * Gates, state and every sum are fp32; out is h rounded once. Results are
 * run-to-run identical.
 */
#define GDN_RECURRENCE_CHUNK 4 /* tokens between two rows of chunk_states */

typedef struct {
    int32_t B, T;        /* batch rows, tokens per row (at most 2^31 - 2^16); with
                            cu_seqlens: B = 1 and T = total packed tokens */
    int32_t N;           /* sequences: B without cu_seqlens, else cu_seqlens has N+1 entries */
    int32_t D;           /* channels (at most 2^30) */
    int32_t dtype;       /* gdn_dtype of x, a, b, out and their gradients */
    int32_t reserved0;
    /* (batch, token) element strides; channel stride is 1 */
    int64_t x_stride_b, x_stride_t;
    int64_t a_stride_b, a_stride_t;
    int64_t b_stride_b, b_stride_t;
} gdn_recurrence_desc;

/* Fill *d for contiguous x, a, b [B,T,D]. packed as in gdn_desc_init. Returns the
 * validation status of the filled descriptor. */
int gdn_recurrence_desc_init(gdn_recurrence_desc *d, int B, int T, int packed, int D, int dtype);

/* Bytes of workspace of the forward (a status word) and of the backward (the
 * status word, partial sums of the parameter gradients, chunk states). */
int gdn_recurrence_workspace_bytes(const gdn_recurrence_desc *d, size_t *bytes);
int gdn_recurrence_backward_workspace_bytes(const gdn_recurrence_desc *d, size_t *bytes);

/*
 * Forward over B rows or packed sequences.
 *   x, a, b        [B,T,D] at their strides
 *   A_log, dt_bias fp32 [D]
 *   cu_seqlens     NULL, or int32 [N+1] (then B == 1); sequences may be empty
 *   initial_state  NULL (zeros) or fp32 [N][D]
 *   out            [B,T,D] contiguous
 *   final_state    NULL or fp32 [N][D]: h after each sequence's last token, its
 *                  initial state (zeros without one) where it is empty
 *   chunk_states   NULL or fp32 [B][ceil(T/4)][D]: the state carried into tokens
 *                  0, 4, 8, ... of each row, for gdn_recurrence_backward
 *   workspace      >= gdn_recurrence_workspace_bytes(), 256-byte aligned;
 *                  gdn_device_status reads its status word
 * x, a, b and out may be NULL when B*T == 0. initial_state and final_state may
 * alias; other outputs must not overlap the inputs. A malformed cu_seqlens sets
 * GDN_ERR_DEVICE_SEQLENS and nothing else is written. Copies into shared memory, and
 * what the CTAs that share a row pass on to one another, are waited for about a second
 * at most (GDN_ERR_DEVICE_TIMEOUT, results invalid).
 */
int gdn_recurrence_forward(const gdn_recurrence_desc *d, const void *x, const void *a, const void *b,
                           const float *A_log, const float *dt_bias, const int32_t *cu_seqlens,
                           const float *initial_state, void *out, float *final_state,
                           float *chunk_states, void *workspace, size_t workspace_bytes,
                           gdn_stream_t stream);

/*
 * Gradients of sum(grad_out * out) + sum(grad_final * final_state).
 *   chunk_states   as written by the forward of the same inputs, or NULL: the call
 *                  then recomputes them in its workspace (one more pass over x, a, b)
 *   grad_out       [B,T,D] contiguous; grad_final NULL (zeros) or fp32 [N][D]
 *   dx, da, db     [B,T,D] contiguous, act dtype
 *   dA_log, ddt_bias  fp32 [D], sums over all tokens in a fixed order
 *   dinitial_state NULL or fp32 [N][D]; grad_final's row where a sequence is empty
 *   workspace      >= gdn_recurrence_backward_workspace_bytes(), 256-byte aligned
 * Outputs are written in full and must not overlap the inputs or each other. A
 * malformed cu_seqlens and a wait that runs out are reported as in the forward.
 * Where g_t = 0 in fp32 (no decay, so no write), the derivative of
 * sqrt(1 - alpha^2) is taken as its limit in a, 0.
 */
int gdn_recurrence_backward(const gdn_recurrence_desc *d, const void *x, const void *a, const void *b,
                            const float *A_log, const float *dt_bias, const int32_t *cu_seqlens,
                            const float *initial_state, const float *chunk_states,
                            const void *grad_out, const float *grad_final, void *dx, void *da,
                            void *db, float *dA_log, float *ddt_bias, float *dinitial_state,
                            void *workspace, size_t workspace_bytes, gdn_stream_t stream);

/*
 * One more token of each of B sequences (d->T == 1, N == B): the state, fp32
 * [B][D], is read and overwritten with h; out [B,1,D] contiguous, which must not
 * overlap the state or the inputs. No workspace.
 */
int gdn_recurrence_step(const gdn_recurrence_desc *d, const void *x, const void *a, const void *b,
                        const float *A_log, const float *dt_bias, float *state, void *out,
                        gdn_stream_t stream);

/*
 * Rotary positions. The first `rot` channels of every head are rotated in pairs
 * (x1, x2) by the angle of the token's position p and the pair's index i:
 *     y1 = scale * (x1 cos - x2 sin),  y2 = scale * (x2 cos + x1 sin),
 * with sin negated for inverse != 0 (the gradient of the rotation, and its undoing
 * when scale is 1). The other channels are copied. The angle is 2 pi times the
 * fraction of p * turns[i] / 2^64: the product wraps in 64 bits, so far positions
 * lose nothing.
 */
typedef enum {
    GDN_ROTARY_HALF = 0,        /* pairs (i, i + rot/2) */
    GDN_ROTARY_INTERLEAVED = 1  /* pairs (2i, 2i + 1) */
} gdn_rotary_layout;
typedef enum {
    GDN_ROTARY_PLAIN = 0,    /* f_i = theta^(-2i/rot) radians per position */
    GDN_ROTARY_LINEAR = 1,   /* f_i / factor */
    GDN_ROTARY_BY_PARTS = 2  /* keep_i f_i + (1 - keep_i) f_i / factor, where keep_i =
                                clamp((r_i - low) / (high - low), 0, 1) and r_i =
                                original * f_i / (2 pi), the pair's turns over the
                                original context */
} gdn_rotary_scaling;

typedef struct {
    int32_t B, T, N;     /* as in gdn_recurrence_desc */
    int32_t Hq, Hk;      /* heads of q and of k; Hk = 0: no k */
    int32_t d;           /* channels per head */
    int32_t rot;         /* rotated channels per head: even, 2..d (at most 32768; a token's
                            channels, (Hq + Hk) d, at most 2^24, tokens below 2^31) */
    int32_t layout;      /* gdn_rotary_layout */
    int32_t inverse;     /* 0 or 1 */
    int32_t dtype;       /* gdn_dtype of q, k and their outputs */
    float scale;         /* 1, or the attention factor of a scaled table */
    int32_t reserved0;
    /* (batch, token) element strides; a token's heads and channels are contiguous */
    int64_t q_stride_b, q_stride_t, k_stride_b, k_stride_t;
    int64_t q_out_stride_b, q_out_stride_t, k_out_stride_b, k_out_stride_t;
} gdn_rotary_desc;

/* Fill *d for contiguous q [B,T,Hq*d], k [B,T,Hk*d] and outputs, rot = d (d - 1
 * where d is odd), half layout, inverse 0, scale 1. Returns the validation status. */
int gdn_rotary_desc_init(gdn_rotary_desc *d, int B, int T, int packed, int Hq, int Hk, int head_dim,
                         int dtype);

/* Host function: the rot/2 table entries f_i / (2 pi) turns per position in units
 * of 2^-64 turns, from fp64 arithmetic, into the HOST array `turns`. factor, low,
 * high and original are read by the scalings that use them. Returns
 * GDN_ERR_INVALID_ARG for an odd or non-positive rot, theta <= 0, factor <= 0,
 * high <= low, original <= 0, or values that leave a frequency not finite. */
int gdn_rotary_table(int rot, double theta, int scaling, double factor, double low, double high,
                     double original, uint64_t *turns);

int gdn_rotary_workspace_bytes(const gdn_rotary_desc *d, size_t *bytes);

/*
 *   q, k           [B,T,H*d] at their strides (k and k_out NULL when Hk == 0)
 *   turns          device uint64 [rot/2] (gdn_rotary_table)
 *   positions      NULL, or int32 [B][T] contiguous: the tokens' positions (any sign)
 *   cu_seqlens     NULL, or int32 [N+1] (then B == 1): without `positions`, a token's
 *                  position counts from its sequence's first token
 *   offsets        NULL, or int32 [N]: added to the positions of sequence n's tokens
 *                  (the length of its cache, for instance); not together with `positions`
 *   q_out, k_out   may be q and k themselves (same strides), else must not overlap them
 *   workspace      >= gdn_rotary_workspace_bytes(), 256-byte aligned (status word). A
 *                  malformed cu_seqlens sets GDN_ERR_DEVICE_SEQLENS and q_out, k_out
 *                  are not written.
 */
int gdn_rotary(const gdn_rotary_desc *d, const void *q, const void *k, const uint64_t *turns,
               const int32_t *positions, const int32_t *cu_seqlens, const int32_t *offsets,
               void *q_out, void *k_out, void *workspace, size_t workspace_bytes,
               gdn_stream_t stream);

/*
 * Group norm with an activation, channels last. For every instance n and group of
 * C/G adjacent channels, mean and (biased) variance over the instance's L positions
 * and the group's channels; then
 *     xh = (x - mean) * rsqrt(var + eps),  z = weight[c] * xh + bias[c],
 *     out = z (GDN_ACT_NONE) or z * sigmoid(z) (GDN_ACT_SILU).
 * L = 1 is the per-token norm of a layer's heads. All arithmetic is fp32; out is
 * rounded once. Results are run-to-run identical.
 */
typedef enum { GDN_ACT_NONE = 0, GDN_ACT_SILU = 1 } gdn_activation;

typedef struct {
    int32_t N, L;          /* instances, positions per instance (either may be 0; L at
                              most 2^31 - 2^16) */
    int32_t C, G;          /* channels (at most 2^24), groups (C % G == 0) */
    int32_t dtype;         /* gdn_dtype of x, out, grad_out, dx */
    int32_t weight_dtype;  /* of weight and bias: dtype, or GDN_F32 */
    int32_t act;           /* gdn_activation */
    float eps;             /* 1e-5 */
    int64_t x_stride_n, x_stride_l; /* element strides of x; channel stride is 1 */
} gdn_group_norm_desc;

/* Fill *d for contiguous x [N,L,C], weight in the act dtype, SiLU, eps 1e-5.
 * Returns the validation status. */
int gdn_group_norm_desc_init(gdn_group_norm_desc *d, int N, int L, int C, int G, int dtype);
int gdn_group_norm_workspace_bytes(const gdn_group_norm_desc *d, size_t *bytes);
int gdn_group_norm_backward_workspace_bytes(const gdn_group_norm_desc *d, size_t *bytes);

/*
 *   x            [N,L,C] at its strides
 *   weight, bias [C] or NULL (ones, zeros)
 *   out          [N,L,C] contiguous
 *   mean, rstd   NULL, or fp32 [N][G]: the statistics, for the backward
 *   workspace    >= gdn_group_norm_workspace_bytes(), 256-byte aligned
 * out must not overlap x. Nothing is written when N*L == 0.
 */
int gdn_group_norm_forward(const gdn_group_norm_desc *d, const void *x, const void *weight,
                           const void *bias, void *out, float *mean, float *rstd, void *workspace,
                           size_t workspace_bytes, gdn_stream_t stream);

/*
 * Gradients of sum(grad_out * out), with mean and rstd from the forward of the same x.
 *   grad_out       [N,L,C] contiguous
 *   dx             [N,L,C] contiguous
 *   dweight, dbias NULL, or fp32 [C] (written also when weight or bias is NULL; zeros
 *                  when N*L == 0)
 *   workspace      >= gdn_group_norm_backward_workspace_bytes(), 256-byte aligned
 * dx must not overlap x or grad_out.
 */
int gdn_group_norm_backward(const gdn_group_norm_desc *d, const void *x, const void *weight,
                            const void *bias, const float *mean, const float *rstd,
                            const void *grad_out, void *dx, float *dweight, float *dbias,
                            void *workspace, size_t workspace_bytes, gdn_stream_t stream);

/*
 * ---------------------------------------------------------------------------
 * Operators of the attention layers that stand between delta rule layers: the
 * norm of every head of q and k together with the rotary positions, and causal
 * softmax attention over a window of recent tokens plus a few first ones, for
 * training, for prefill and for single tokens over a cache of fixed size. The
 * conventions of the operators above hold; the definitions stand here in full.
 */

/*
 * Head norm and rotary positions in one pass. For every token and head of q (of k),
 * x the head's d channels and w its weight [d] (all heads of q share one weight, all
 * heads of k another):
 *     xh = x * rsqrt(mean_c x^2 + eps),  z = xh * w,  y = rotary(z),
 * the rotation of gdn_rotary (positions, layouts, tables, scale). All arithmetic is
 * fp32; y is rounded once. Results are run-to-run identical.
 */
typedef struct {
    gdn_rotary_desc rotary; /* sizes, layout and strides as in gdn_rotary; inverse 0, d at most 1024 */
    int32_t weight_dtype;   /* of q_weight and k_weight: rotary.dtype, or GDN_F32 */
    float eps;              /* 1e-6 */
} gdn_norm_rotary_desc;

/* Fill *d as gdn_rotary_desc_init does, weights in the act dtype, eps 1e-6. */
int gdn_norm_rotary_desc_init(gdn_norm_rotary_desc *d, int B, int T, int packed, int Hq, int Hk,
                              int head_dim, int dtype);
int gdn_norm_rotary_workspace_bytes(const gdn_norm_rotary_desc *d, size_t *bytes);
int gdn_norm_rotary_backward_workspace_bytes(const gdn_norm_rotary_desc *d, size_t *bytes);

/*
 *   q, k, turns, positions, cu_seqlens, offsets, q_out, k_out, workspace
 *                       as in gdn_rotary (in place allowed: the same strides then)
 *   q_weight, k_weight  [d] or NULL (ones)
 */
int gdn_norm_rotary_forward(const gdn_norm_rotary_desc *d, const void *q, const void *k,
                            const void *q_weight, const void *k_weight, const uint64_t *turns,
                            const int32_t *positions, const int32_t *cu_seqlens,
                            const int32_t *offsets, void *q_out, void *k_out, void *workspace,
                            size_t workspace_bytes, gdn_stream_t stream);

/*
 * Gradients of sum(grad_q * q_out) + sum(grad_k * k_out); q and k are the forward's inputs.
 *   grad_q, grad_k      [B,T,H*d] at the descriptor's q_out and k_out strides
 *   dq, dk              [B,T,H*d] contiguous (dk NULL when Hk == 0); must not overlap inputs
 *   dq_weight, dk_weight  NULL, or fp32 [d]: sums over all tokens and heads in a fixed
 *                       order (written also when the weight is NULL; zeros when B*T == 0)
 *   workspace           >= gdn_norm_rotary_backward_workspace_bytes(), 256-byte aligned.
 *                       A malformed cu_seqlens sets GDN_ERR_DEVICE_SEQLENS and nothing
 *                       else is written.
 */
int gdn_norm_rotary_backward(const gdn_norm_rotary_desc *d, const void *q, const void *k,
                             const void *q_weight, const void *k_weight, const uint64_t *turns,
                             const int32_t *positions, const int32_t *cu_seqlens,
                             const int32_t *offsets, const void *grad_q, const void *grad_k,
                             void *dq, void *dk, float *dq_weight, float *dk_weight,
                             void *workspace, size_t workspace_bytes, gdn_stream_t stream);

/*
 * Window attention. A sequence has Lk keys and Lq queries, the queries being its last
 * Lq positions: query i stands at position p = Lk - Lq + i. It sees the keys
 *     j <= p  with  p - j < window  or  j < sinks,
 * that is the `window` most recent tokens, itself among them, and the sequence's first
 * `sinks` tokens, which stay visible. Head h of q reads head h / (Hq/Hk) of k and v:
 *     s_j = scale * q . k_j,  P = softmax over the keys seen,  out = sum_j P_j v_j,
 *     lse = log sum_j exp(s_j).
 * A query that sees nothing (p < 0, where Lq > Lk) gets out = 0 and lse = -inf.
 * Scores, softmax statistics and every sum are fp32; with 16-bit types the tensor-core
 * kernels round P, and in the backward P and the scores' gradients, to that type as
 * operands of their products, fp16 ones times powers of two that keep them in its range
 * (in the backward by the largest finite rows of grad_out and v of a sequence and head of k). Results are run-to-run identical. What a query does not
 * see has no influence on its output, also where it is infinite or NaN; in the backward
 * this holds between sequences (inside one, a NaN may reach neighbouring gradients).
 */
typedef struct {
    int32_t B;           /* batch rows; with cu_seqlens B = 1 */
    int32_t Tq, Tk;      /* queries and keys per row; packed: totals. At most 2^31 - 2^16 */
    int32_t N;           /* sequences: B without cu_seqlens, else cu_seqlens has N+1 entries */
    int32_t Hq, Hk;      /* heads of q, of k and v (Hq % Hk == 0) */
    int32_t d;           /* channels per head, 1..256 */
    int32_t window;      /* >= 1; at least Tk: plain causal attention */
    int32_t sinks;       /* >= 0 */
    int32_t slots;       /* cache calls: slots per head, sinks + window to 2^31 - 2^16 */
    int32_t dtype;       /* gdn_dtype of q, k, v, out, their gradients and the caches */
    float scale;         /* 1/sqrt(d) */
    /* (batch, token) element strides; a token's heads and channels are contiguous */
    int64_t q_stride_b, q_stride_t, k_stride_b, k_stride_t, v_stride_b, v_stride_t;
} gdn_window_attention_desc;

/* Fill *d for contiguous q [B,Tq,Hq*d], k, v [B,Tk,Hk*d], scale 1/sqrt(d), slots
 * sinks + window. packed as in gdn_desc_init. Returns the validation status. */
int gdn_window_attention_desc_init(gdn_window_attention_desc *d, int B, int Tq, int Tk, int packed,
                                   int Hq, int Hk, int head_dim, int window, int sinks, int dtype);
int gdn_window_attention_workspace_bytes(const gdn_window_attention_desc *d, size_t *bytes);
int gdn_window_attention_backward_workspace_bytes(const gdn_window_attention_desc *d, size_t *bytes);
int gdn_window_attention_step_workspace_bytes(const gdn_window_attention_desc *d, size_t *bytes);
int gdn_window_cache_write_workspace_bytes(const gdn_window_attention_desc *d, size_t *bytes);

/* Which kernels serve *d in the forward and backward, given aligned tensors: 0 = fp32
 * CUDA-core kernels, 1 = tcgen05 tensor-core kernels (16-bit types, d a multiple of 8 up
 * to 128, every q, k and v base 16-byte aligned and every stride a multiple of 8). */
int gdn_window_attention_kernel_kind(const gdn_window_attention_desc *d);

/*
 *   q, k, v        at their strides
 *   cu_seqlens     NULL, or int32 [N+1] offsets of the queries (then B == 1)
 *   cu_seqlens_k   NULL (the same as cu_seqlens; Tk == Tq then), or int32 [N+1] offsets of
 *                  the keys
 *   out            [B,Tq,Hq*d] contiguous
 *   lse            NULL, or fp32 [Hq][B*Tq]: for the backward
 *   workspace      >= gdn_window_attention_workspace_bytes(), 256-byte aligned;
 *                  gdn_device_status reads its status word. Malformed offsets set
 *                  GDN_ERR_DEVICE_SEQLENS and nothing else is written. Waits for copies
 *                  and products give up after about a second (GDN_ERR_DEVICE_TIMEOUT).
 * out and lse must not overlap the inputs or each other.
 */
int gdn_window_attention_forward(const gdn_window_attention_desc *d, const void *q, const void *k,
                                 const void *v, const int32_t *cu_seqlens,
                                 const int32_t *cu_seqlens_k, void *out, float *lse,
                                 void *workspace, size_t workspace_bytes, gdn_stream_t stream);

/*
 * Gradients of sum(grad_out * out), with out and lse of the forward on the same inputs.
 *   out, grad_out  [B,Tq,Hq*d] contiguous
 *   dq             [B,Tq,Hq*d] contiguous;  dk, dv  [B,Tk,Hk*d] contiguous: written in
 *                  full, each rounded once. They must not overlap the inputs or each other.
 *   workspace      >= gdn_window_attention_backward_workspace_bytes(), 256-byte aligned;
 *                  status as in the forward
 */
int gdn_window_attention_backward(const gdn_window_attention_desc *d, const void *q, const void *k,
                                  const void *v, const void *out, const float *lse,
                                  const void *grad_out, const int32_t *cu_seqlens,
                                  const int32_t *cu_seqlens_k, void *dq, void *dk, void *dv,
                                  void *workspace, size_t workspace_bytes, gdn_stream_t stream);

/*
 * The cache (Hk at most 65535): per sequence and head `slots` rows of keys and of values,
 * k_cache, v_cache [N][Hk][slots][d] contiguous, whatever the sequence's length. Position
 * p is held in slot p for p < sinks, else in slot sinks + (p - sinks) % (slots - sinks),
 * where it stays until a later position takes the slot over. lengths, int32 [N], counts
 * the positions that a sequence has had before the call, 0 .. 2^31 - 2; the call does not
 * change it (the layers of a model share it). A sequence whose length is negative takes
 * no part: its cache is left as it is.
 *
 * gdn_window_cache_write puts tokens at positions lengths[n], lengths[n] + 1, ... of each
 * sequence n, those that a later one of the same call would replace left out.
 *   k, v           [B,Tk,Hk*d] at their strides (Tq, Hq, scale and q's strides have no effect, but
 *                  have to be valid, as gdn_window_attention_desc_init fills them: Hq % Hk == 0)
 *   cu_seqlens     NULL, or int32 [N+1] (then B == 1): offsets into k and v
 *   workspace      >= gdn_window_cache_write_workspace_bytes(), 256-byte aligned (status
 *                  word; a malformed cu_seqlens writes nothing else)
 */
int gdn_window_cache_write(const gdn_window_attention_desc *d, const void *k, const void *v,
                           const int32_t *cu_seqlens, const int32_t *lengths, void *k_cache,
                           void *v_cache, void *workspace, size_t workspace_bytes,
                           gdn_stream_t stream);

/*
 * One more token of each of B sequences (d->Tq == d->Tk == 1, N == B): k and v are written
 * into the caches at position lengths[n], and the query attends to the cache with the mask
 * of the window attention at that position. Positions never written must not be counted in
 * lengths.
 *   q [B,1,Hq*d], k, v [B,1,Hk*d] at their batch strides
 *   out            [B,1,Hq*d] contiguous; zeros for a sequence that takes no part
 *   workspace      >= gdn_window_attention_step_workspace_bytes(), 256-byte aligned; calls
 *                  that share one must not overlap on the GPU
 * The result is that of gdn_window_attention_forward on the whole sequence's last token
 * (another order of the sums).
 */
int gdn_window_attention_step(const gdn_window_attention_desc *d, const void *q, const void *k,
                              const void *v, const int32_t *lengths, void *k_cache, void *v_cache,
                              void *out, void *workspace, size_t workspace_bytes,
                              gdn_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* GDN_H */

/*
 * moe.h -- C ABI of the latent mixture-of-experts layer on AMD MI355X (gfx950).
 *
 * The layer (one MoE layer of the 816B-A42B "Muse Spark Open" model):
 *   1. an fp32 router scores every expert for each token and keeps the top K
 *      ("Muse Spark Open on Gaudi 2", section "What was built": fp32 router,
 *      256 experts, top 8);
 *   2. the routes are grouped by expert;
 *   3. one pooler shared by all experts projects each token from the hidden
 *      width H to the latent width L ("Soporte de dia 0 para Muse Spark Open
 *      en vLLM", section "Arquitectura del modelo", paragraph "MoE latente");
 *   4. every (token, route) pair is its own row through its expert's MXFP4
 *      SwiGLU FFN, W4A16: 4-bit E2M1 weights with E8M0 block scales, bf16
 *      activations ("Muse Spark Open on Gaudi 2", sections "What was built"
 *      and "The latent MoE: A' with a per-expert norm");
 *   5. each route row gets the post-expert RMS norm, then the rows are
 *      multiplied by the router weights and summed in fp32 (same section);
 *   6. the shared unpooler projects the sum from L back to H (same section).
 *
 * Conventions for every entry point:
 *  - Device pointers unless stated otherwise; bf16 values are passed as their
 *    16-bit patterns (uint16_t). All matrices are row-major.
 *  - Ownership: the caller allocates and owns every buffer and the stream.
 *    The library allocates no memory, keeps no state between calls (apart
 *    from the thread-local last HIP error) and never synchronises the host:
 *    work is enqueued on `hip_stream` (a hipStream_t; NULL = default stream),
 *    so calls can be captured into a HIP graph.
 *  - Errors: every entry point returns an int status, MOE_OK (0) or a
 *    negative MOE_E* code. Invalid arguments are reported before anything is
 *    enqueued, and outputs are left untouched. MOE_EHIP means a launch
 *    failed; moe_last_hip_error() returns the HIP error code.
 *  - Inputs, outputs and the workspace must not overlap. T == 0 is a no-op
 *    returning MOE_OK. Outputs are fully overwritten.
 *  - Routing and the permutation are deterministic (bit-identical across
 *    runs); the output does not depend on the workspace contents. (For
 *    T <= 8 the first 256 bytes of the workspace hold a generation word that
 *    each call advances on the device, so that a call, or a replay of a
 *    captured graph, recognises its own router logits among stale words;
 *    any initial contents work, and calls sharing a workspace must not
 *    overlap, as for every other buffer of it.)
 *
 * Supported shapes (else MOE_EUNSUPPORTED): hidden, latent and inter are
 * multiples of 128, at least 128, latent <= 8192, hidden and inter <= 65536;
 * 1 <= n_experts <= 256; 1 <= top_k <= min(8, n_experts);
 * T * top_k < 2^28. Pointers must be 16-byte aligned (MOE_EALIGN), unless an
 * entry point states another alignment.
 */
#ifndef MOE_H
#define MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_OK 0
#define MOE_EINVAL (-1)       /* null pointer, negative size, bad eps or flag   */
#define MOE_EUNSUPPORTED (-2) /* dims outside the supported shapes above        */
#define MOE_EALIGN (-3)       /* a pointer (or row pitch) is not aligned, 16 bytes unless stated otherwise */
#define MOE_EWORKSPACE (-4)   /* workspace smaller than moe_workspace_bytes()   */
#define MOE_EHIP (-5)         /* a HIP launch failed (see moe_last_hip_error)   */

typedef struct {
  int32_t hidden;          /* H: width of the layer input and output (8192)          */
  int32_t latent;          /* L: width after the pooler, the experts' width (4096)    */
  int32_t inter;           /* I: SwiGLU intermediate width of each expert (4096)      */
  int32_t n_experts;       /* E: routed experts (256)                                  */
  int32_t top_k;           /* K: experts per token (8)                                 */
  float norm_eps;          /* eps inside the post-expert RMS norm's square root (1e-6) */
  int32_t gain_per_expert; /* 0: one norm gain [L] for all experts; 1: gain [E][L]     */
  int32_t expert_format;   /* MOE_FMT_MXFP4 or MOE_FMT_NVFP4                           */
  int32_t expert_split_rows; /* the expert projections' two loops (below); 0: default */
} moe_dims;

/* expert_split_rows: how the expert projections treat experts with few
 * routes when the routes average at least 16 per expert (otherwise every
 * expert already runs on the streaming kernels). "RadixArk team serves
 * Meta's Muse Spark Open on one TPU host", section "Changes to attention
 * and expert processing": many-request decode steps under random routing
 * ran faster once the expert work was split into two loops; the page does
 * not say which, and here the two loops are the experts' two row regimes:
 *   n in 1..16: experts with at most n routes stream their weights once for
 *      all their rows (HBM-bound kernels), the others run on MFMA row tiles
 *      (a second launch per projection);
 *   -1: one loop, every expert on the row tiles;
 *   0: the library's choice.
 * Other values return MOE_EINVAL. Results are within the same bounds either
 * way (the two kernels sum in different orders, so the bits may differ). */

/* Expert weight formats. Both store E2M1 codes as below. MXFP4: one E8M0
 * scale byte per 32 elements ([rows][K/32]). NVFP4 (public NVIDIA format;
 * "Soporte de día 0 para Muse Spark Open en vLLM", section "Aspectos
 * destacados": the model ships in NVFP4): one OCP E4M3 scale byte per 16
 * elements ([rows][K/16]) times one fp32 scale per stored tensor and expert
 * (w13_global, w2_global). */
#define MOE_FMT_MXFP4 0
#define MOE_FMT_NVFP4 1

/* Layer weights, as stored (no repacking step). 4-bit expert tensors: byte j
 * of a code row holds element 2j in bits 0..3 and element 2j+1 in bits 4..7
 * (E2M1: sign, 2 exponent bits with bias 1, 1 mantissa bit). MXFP4: one E8M0
 * scale byte (value 2^(b-127)) covers 32 consecutive elements of a row along
 * the reduction dimension. NVFP4: one E4M3 scale byte covers 16, and the
 * tensor's fp32 scale multiplies every element. */
typedef struct {
  const float *router;          /* [E][H] fp32                                     */
  const uint16_t *pooler;       /* [L][H] bf16: lat = x . pooler^T                 */
  const uint8_t *w13_codes;     /* [E][2I][L/2]: rows 0..I-1 gate, I..2I-1 up      */
  const uint8_t *w13_scales;    /* [E][2I][L/32] (NVFP4: [E][2I][L/16])            */
  const uint8_t *w2_codes;      /* [E][L][I/2]: down projection                    */
  const uint8_t *w2_scales;     /* [E][L][I/32] (NVFP4: [E][L][I/16])              */
  const uint16_t *norm_gain;    /* [L] or [E][L] bf16 (see gain_per_expert)        */
  const uint16_t *unpooler;     /* [H][L] bf16: out = y . unpooler^T               */
  const float *w13_global;      /* NVFP4: [E] fp32 scale of each expert's W13      */
  const float *w2_global;       /* NVFP4: [E] fp32 scale of each expert's W2       */
} moe_weights;

/* Token counts: T * H * 2, T * latent * 2 and T * top_k * inter * 2 bytes
 * must each be below 2^31 (T <= 32767 at H 8192, L 4096, K 8, I 4096);
 * larger T returns MOE_EUNSUPPORTED (split the batch).
 *
 * Bytes of device workspace needed by moe_route and moe_latent_forward for
 * any T <= max_tokens. Returns 0 if the dims are invalid or unsupported. */
size_t moe_workspace_bytes(const moe_dims *dims, int32_t max_tokens);

/*
 * moe_route -- steps 1 and 2 for T tokens (router logits, top-K with router
 * weights, grouping of the routes by expert).
 *   x              [T][H] bf16      layer input (the router reads the full
 *                                   H-wide input, converted exactly to fp32)
 *   router         [E][H] fp32
 *   topk_ids       [T][K] int32     out: experts in rank order: larger logit
 *                                   first, equal logits (-0 == +0) by lower
 *                                   id, NaN after every number
 *   topk_w         [T][K] fp32      out: softmax over the K selected logits
 *   expert_offsets [E+1]  int32     out: exclusive prefix sum of the number
 *                                   of routes per expert; [E] = T*K
 *   sorted_routes  [T*K]  int32     out: route ids r = t*K + k grouped by
 *                                   expert, ascending r within an expert
 *   logits_out     [T][E] fp32      out, optional (NULL): the router logits,
 *                                   each the fp32 rounding of the exact sum
 *                                   (accumulated in fp64)
 */
int moe_route(const moe_dims *dims, int32_t T, const uint16_t *x,
              const float *router, int32_t *topk_ids, float *topk_w,
              int32_t *expert_offsets, int32_t *sorted_routes,
              float *logits_out, void *workspace, size_t workspace_bytes,
              void *hip_stream);

/*
 * moe_latent_forward -- the whole layer for T tokens:
 *   out[t] = bf16( unpooler . bf16( sum_k w[t][k] * rmsnorm_e(row[t][k]) ) )
 *   row[t][k] = W2_e . bf16( silu(W13gate_e . lat[t]) * (W13up_e . lat[t]) )
 *   lat[t] = bf16( pooler . x[t] ),   e = topk_ids[t][k]
 * with rmsnorm_e(v) = v / sqrt(mean(v^2) + eps) * gain (gain[e] if per expert).
 *   x   [T][H] bf16,   out [T][H] bf16 (out)
 * Intermediates (router logits, routes, lat, h, route rows, y) live in the
 * workspace; moe_workspace_view() locates them.
 */
int moe_latent_forward(const moe_dims *dims, int32_t T, const uint16_t *x,
                       const moe_weights *weights, uint16_t *out,
                       void *workspace, size_t workspace_bytes,
                       void *hip_stream);

/*
 * moe_latent_forward_routed -- the same layer with the routing given by the
 * caller (routing replay: "Soporte de día 0 para Muse Spark Open en vLLM",
 * section "Aprendizaje por refuerzo en vLLM", where the trainer reuses the
 * rollout's MoE routing). Steps 1 and 2 are skipped; steps 3 to 8 run as in
 * moe_latent_forward with:
 *   topk_ids [T][K] int32  device: the experts of each token, each in [0, E).
 *                          A token may list an expert more than once (each
 *                          listing is its own route row). Ids outside
 *                          [0, E) are not reported: they are clamped into
 *                          range, so the result is unspecified but no
 *                          access leaves the weights.
 *   topk_w   [T][K] fp32   device: router weights, used as given (no
 *                          renormalisation).
 * weights->router is not read (may be NULL). The grouping and the clamped
 * ids are left in the workspace as for moe_latent_forward (views OFFSETS,
 * SORTED, IDS); the weights view is not written. Same errors as
 * moe_latent_forward.
 */
int moe_latent_forward_routed(const moe_dims *dims, int32_t T, const uint16_t *x,
                              const int32_t *topk_ids, const float *topk_w,
                              const moe_weights *weights, uint16_t *out,
                              void *workspace, size_t workspace_bytes,
                              void *hip_stream);

/*
 * moe_block_forward -- the layer inside its block: the sandwich norms and the
 * residual ("Soporte de día 0 para Muse Spark Open en vLLM", section
 * "Arquitectura del modelo": out = x + post_norm(F(norm(x))); section
 * "Nvidia": the router is fed by the norm's fp32 output):
 *   n      = resid[t] / sqrt(mean(resid[t]^2) + block_eps) * pre_gain
 *            (fp64; the router reads fp32(n), the pooler bf16(n))
 *   f[t]   = the layer of moe_latent_forward on that input
 *   out[t] = bf16( resid[t] + f[t] / sqrt(mean(f[t]^2) + block_eps) * post_gain )
 *   resid     [T][H] bf16   the residual stream (the block's input)
 *   pre_gain  [H]    bf16   gain of the norm before the layer
 *   post_gain [H]    bf16   gain of the norm after the layer
 *   block_eps        fp32   eps inside both square roots (>= 0)
 *   out       [T][H] bf16   out; may be the same buffer as resid
 * The workspace must hold moe_block_workspace_bytes(dims, T) bytes; it also
 * holds the layer's intermediates (moe_workspace_view, including the views
 * NORM_F32, NORM_BF16 and LAYER_OUT). Same errors as moe_latent_forward, and
 * MOE_EINVAL for a null gain or a negative or non-finite block_eps.
 */
size_t moe_block_workspace_bytes(const moe_dims *dims, int32_t max_tokens);
int moe_block_forward(const moe_dims *dims, int32_t T, const uint16_t *resid,
                      const uint16_t *pre_gain, const uint16_t *post_gain,
                      float block_eps, const moe_weights *weights, uint16_t *out,
                      void *workspace, size_t workspace_bytes, void *hip_stream);

/* Same as moe_latent_forward, and additionally times each step with HIP
 * events recorded by the step's kernel launch itself (hipExtLaunchKernel),
 * so nothing else is added to the stream. stage_events: NULL, or an array of
 * 2 * MOE_N_STAGES hipEvent_t created by the caller: events 2i and 2i+1 mark
 * the start and end of step i; NULL entries are skipped. A step that needs
 * no kernel for the given T records its two events back to back. For
 * T <= 16 the router and the pooler share one launch, timed as step 0
 * (step 3 then has no kernel), and top-k and grouping share one launch,
 * timed as step 1. */
#define MOE_N_STAGES 8 /* router, top-k, permute, pool, gate/up, down, combine, unpool */
int moe_latent_forward_timed(const moe_dims *dims, int32_t T,
                             const uint16_t *x, const moe_weights *weights,
                             uint16_t *out, void *workspace,
                             size_t workspace_bytes, void *hip_stream,
                             void *const *stage_events);

/* Argument checks of moe_route / moe_latent_forward without enqueuing
 * anything (callable without a GPU). Same arguments and return codes. */
int moe_route_validate(const moe_dims *dims, int32_t T, const uint16_t *x,
                       const float *router, const int32_t *topk_ids,
                       const float *topk_w, const int32_t *expert_offsets,
                       const int32_t *sorted_routes, const float *logits_out,
                       const void *workspace, size_t workspace_bytes);
int moe_latent_forward_routed_validate(const moe_dims *dims, int32_t T,
                                       const uint16_t *x, const int32_t *topk_ids,
                                       const float *topk_w, const moe_weights *weights,
                                       const uint16_t *out, const void *workspace,
                                       size_t workspace_bytes);
int moe_block_forward_validate(const moe_dims *dims, int32_t T, const uint16_t *resid,
                               const uint16_t *pre_gain, const uint16_t *post_gain,
                               float block_eps, const moe_weights *weights,
                               const uint16_t *out, const void *workspace,
                               size_t workspace_bytes);
int moe_latent_forward_validate(const moe_dims *dims, int32_t T,
                                const uint16_t *x, const moe_weights *weights,
                                const uint16_t *out, const void *workspace,
                                size_t workspace_bytes);

/* Location of an intermediate inside the workspace after moe_latent_forward
 * for T tokens: byte offset and size. Returns MOE_EINVAL for an unknown id.
 *   MOE_VIEW_LOGITS  [T][E] fp32       MOE_VIEW_IDS    [T][K] int32
 *   MOE_VIEW_WEIGHTS [T][K] fp32       MOE_VIEW_OFFSETS [E+1] int32
 *   MOE_VIEW_SORTED  [T*K] int32       MOE_VIEW_LATENT [T][L] bf16
 *   MOE_VIEW_H       [T*K][I] bf16, row i belongs to route sorted_routes[i]
 *   MOE_VIEW_ROWS    [T*K][L] fp32, route-major (r = t*K + k)
 *   MOE_VIEW_Y       [T][L] bf16 (normed, weighted sum); not written when
 *                    MOE_VIEW_ROWS_BF16 has a nonzero size
 *   MOE_VIEW_ROWS_BF16 [T*K][L] bf16, route-major: bf16(gain * row), the
 *                    unpooler's input when few route rows (T*K <= 16 whose
 *                    latent rows fit 72 KiB, on the streaming expert path;
 *                    with NVFP4 experts one token only) let one launch
 *                    take the post-norm, the weighted sum and the
 *                    unpooler: out[t] = bf16(sum over the token's
 *                    routes of w / sqrt(mean(row^2) + eps) * (unpooler .
 *                    bf16(gain * row))), the weighted sum after the
 *                    products ("Muse Spark Open on Gaudi 2", section "The
 *                    latent MoE: A' with a per-expert norm"; both are
 *                    linear); 0 bytes otherwise (the same for
 *                    moe_latent_forward_persistent). */
#define MOE_VIEW_LOGITS 0
#define MOE_VIEW_IDS 1
#define MOE_VIEW_WEIGHTS 2
#define MOE_VIEW_OFFSETS 3
#define MOE_VIEW_SORTED 4
#define MOE_VIEW_LATENT 5
#define MOE_VIEW_H 6
#define MOE_VIEW_ROWS 7
#define MOE_VIEW_Y 8
#define MOE_VIEW_NORM_F32 9   /* moe_block_forward: [T][H] fp32 pre-norm output */
#define MOE_VIEW_NORM_BF16 10 /* moe_block_forward: [T][H] bf16 pre-norm output */
#define MOE_VIEW_LAYER_OUT 11 /* moe_block_forward: [T][H] bf16 layer output    */
/* The words that carry over between calls (256 bytes at offset 0 whatever
 * T): uint32 [0] the generation word of the routing done inside the router
 * launch (T <= 8) and of the persistent decode layer, advanced by exactly
 * one per such call; [1] status bits, bit 0 set if a router workgroup ever
 * gave up its bounded wait for that routing, bit 1 if a wait of the
 * persistent decode layer gave up (the call's output is then not valid; not
 * expected to happen; bits 2-4 name the wait: routing flag, release, tagged
 * logits); [2] the persistent
 * layer's routing flag; [3] its workgroup count; [8]-[12] and [16]-[21] its
 * last call's clock stamps (the 100 MHz constant clock, low 32 bits):
 * routing done and barriers 1-4 released; workgroup 0's start and the end
 * of its five phases (with few route rows, see MOE_VIEW_ROWS_BF16: barriers
 * 1-3, and the start and end of the unpooler's phase, which also takes the
 * post-norm and the weighted sum, in place of phases 4 and 5). */
#define MOE_VIEW_SYNC 12
#define MOE_VIEW_ROWS_BF16 13
int moe_workspace_view(const moe_dims *dims, int32_t T, int32_t which,
                       size_t *offset, size_t *bytes);

/* The same layer for one or two tokens in a single launch: the persistent
 * decode layer ("RadixArk team serves Meta's Muse Spark Open on one TPU
 * host", section "A single program for a serving step"). One grid, sized to
 * what the device holds at once, runs the router and pooler, the routing,
 * gate/up, down, the post-norm and weighted sum, and the unpooler as phases
 * separated by barriers between its workgroups (with few route rows the
 * post-norm and the weighted sum run in the unpooler's phase, as in
 * moe_latent_forward); every workgroup issues its next weights before it
 * waits. Same arguments, workspace and results as moe_latent_forward (the
 * workspace views hold the same intermediates).
 *  - T > 2, T * top_k > 64, or shapes outside what its phases are compiled
 *    for (hidden and latent multiples of 4096 with inter a multiple of
 *    2048, as the real shape is) return MOE_EUNSUPPORTED before anything is
 *    enqueued.
 *  - It assumes every workgroup of its grid is scheduled while the others
 *    wait: other kernels running on the device at the same time (another
 *    stream, another process) can keep part of the grid out; the bounded
 *    waits then give up, bit 1 of the MOE_VIEW_SYNC status word is set and
 *    the output is not valid. */
int moe_latent_forward_persistent(const moe_dims *dims, int32_t T, const uint16_t *x,
                                  const moe_weights *weights, uint16_t *out, void *workspace,
                                  size_t workspace_bytes, void *hip_stream);

/* moe_latent_forward for callers that cannot allocate device memory (code
 * under HIP graph capture that must not allocate, tight serving loops,
 * harnesses that forbid hipMalloc): the same layer and the same kernels,
 * with the workspace taken from a file-scope device array of
 * MOE_NOALLOC_SCRATCH_BYTES that each GPU the library runs on holds until
 * the process ends. The caller still passes the inputs, the weights and
 * `out`. Allocates nothing: on the first call on a device (the current one)
 * the array's device address is looked up once (hipGetSymbolAddress) and
 * kept for that device.
 *  - T with moe_workspace_bytes(dims, T) > MOE_NOALLOC_SCRATCH_BYTES returns
 *    MOE_EWORKSPACE before anything is enqueued (at the real shape,
 *    H 8192, L 4096, E 256, K 8, I 4096: T <= 55, decode and verify).
 *  - Every call on one GPU shares that GPU's array, which keeps the last
 *    call's contents (the layer needs no cleared workspace): calls that
 *    overlap on one GPU (several streams or host threads) race, and the
 *    caller must order them.
 *  - A device index beyond 63 returns MOE_EUNSUPPORTED; other errors as
 *    moe_latent_forward. */
#define MOE_NOALLOC_SCRATCH_BYTES (32u << 20)
int moe_latent_forward_noalloc(const moe_dims *dims, int32_t T, const uint16_t *x,
                               const moe_weights *weights, uint16_t *out, void *hip_stream);

/*
 * 8-bit rows and their products: E4M3 codes (OCP FP8 "fn": largest value
 * 448, no infinities) with one fp32 scale per 128 consecutive values of a
 * row, and weights with one fp32 scale per 128 x 128 block. They stand
 * beside the layer's bf16 pooler and unpooler (moe_fp8_linear) and its FP4
 * experts (moe_fp8_grouped), for weights stored that way.
 *
 * Widths (cols, K) are multiples of 16 up to 65536 and need not be multiples
 * of 128: the last scale covers what is left. N up to 65536. Rows below
 * 2^28. Codes, x and weights 16-byte aligned, rows of x 16-byte aligned
 * (pitches in elements, at most 2^22; MOE_EALIGN); scales, offsets, indices
 * and out need the alignment of their type only. Zero rows are a no-op.
 *
 * moe_fp8_quantize: x [rows][cols] (pitch ldx) of x_type to
 *   codes  [rows][cols]            e4m3(x * (448 / amax)), nearest even
 *   scales [rows][ceil(cols/128)]  amax / 448
 * amax: the largest finite |x| of the group, at least 2^-90. NaN and
 * infinities become NaN codes and do not raise the scale.
 * moe_fp8_swiglu: the same of h = silu(gate) * up in fp32; a row of gate_up
 * holds inter gate values, then inter up values (the rows the gate/up
 * product of w13 gives).
 */
#define MOE_TYPE_BF16 0
#define MOE_TYPE_F32 1
int moe_fp8_quantize(int32_t rows, int32_t cols, const void *x, int64_t ldx,
                     int32_t x_type, uint8_t *codes, float *scales,
                     void *hip_stream);
int moe_fp8_swiglu(int32_t rows, int32_t inter, const void *gate_up, int64_t ld,
                   int32_t type, uint8_t *codes, float *scales,
                   void *hip_stream);

/* moe_fp8_linear: out[t][n] = sum over blocks b of 128 of
 *     x_scales[t][b] * w_scales[n/128][b] * sum_{k in b} x[t][k] * w[n][k]
 *   x [T][K] codes (pitch ldx), x_scales [T][ceil(K/128)],
 *   w [N][K] codes, w_scales [ceil(N/128)][ceil(K/128)],
 *   out [T][N] (pitch ldo) of out_type, rounded once from an fp32 sum of the
 *   blocks. Within a block an fp32 out sums in fp32, and so does a bf16 out of
 *   up to 16 rows. A bf16 out of more takes the E4M3 matrix instruction's own
 *   sum, which drops from each eight neighbouring products what lies 2^-14 below
 *   the largest of them, up to 7 * 2^-14 of it: inside its final rounding unless
 *   the terms cancel each other, when it may be off in all its bits. With
 *   MOE_SUM_F32 added to out_type a bf16 out sums in fp32 always, at 1.1 times
 *   the time for tens of rows and up to 2.1 times for thousands. (The order of
 *   fp32 additions goes by the sizes.) */
#define MOE_SUM_F32 0x100
int moe_fp8_linear(int32_t T, int32_t N, int32_t K, const uint8_t *x,
                   int64_t ldx, const float *x_scales, const uint8_t *w,
                   const float *w_scales, void *out, int64_t ldo,
                   int32_t out_type, void *hip_stream);

/* moe_fp8_grouped: the same product for every expert over its own rows:
 * output rows offsets[e] .. offsets[e+1]-1 against expert e's weights.
 *   offsets   [n_experts+1] int32, device (moe_route's expert_offsets);
 *             rows outside [offsets[0], offsets[n_experts]) are left as they
 *             were. Offsets that decrease or leave [0, rows] give unspecified
 *             rows but no access outside the buffers.
 *   row_index [rows] int32, device, or NULL: output row i reads row
 *             row_index[i] / index_div of x (moe_route's sorted_routes with
 *             index_div = top_k: each route its token's row; an index outside
 *             x is clamped into it). NULL: row i, index_div 1, x_rows >= rows.
 *   x [x_rows][K], x_scales [x_rows][ceil(K/128)], w [E][N][K],
 *   w_scales [E][ceil(N/128)][ceil(K/128)], out [rows][N].
 * n_experts <= 256; with row_index x_rows * ldx < 2^31. A bf16 out sums by
 * either of moe_fp8_linear's two ways, by the sizes, without MOE_SUM_F32. */
int moe_fp8_grouped(int32_t rows, int32_t n_experts, int32_t N, int32_t K,
                    const int32_t *offsets, const int32_t *row_index,
                    int32_t index_div, int32_t x_rows, const uint8_t *x,
                    int64_t ldx, const float *x_scales, const uint8_t *w,
                    const float *w_scales, void *out, int64_t ldo,
                    int32_t out_type, void *hip_stream);

/*
 * moe_balance_loss -- how evenly the router spreads its tokens, from what
 * moe_route gives, and moe_balance_loss_backward -- the gradient of the
 * router logits, for a trainer.
 *   p = softmax(logits[t]), lse[t] = log(sum_e exp(logits[t][e])),
 *   c_e = routes to expert e, N = tokens that count,
 *   f_e = E * c_e / (K * N), P_e = sum_t p[t][e] / N
 *   losses[0] = sum_e f_e * P_e   (1 when every expert gets the same)
 *   losses[1] = sum_t lse[t]^2 / N
 *   logits     [T][E] fp32, 16-byte aligned
 *   topk_ids   [T][K] int32; ids outside [0, E) are not counted
 *   token_mask [T] uint8 or NULL: tokens with 0 do not count
 *   counts     [E+1] int32 out: c_e, then N
 *   losses     [2] fp32 out
 * Tokens whose logits are all -inf do not count either. With none that
 * counts (also T == 0) counts and losses are written as zeros. The same from
 * run to run, bit for bit. Whatever T is, at most about a hundred additions of
 * one sum are in fp32 (the rest in 64 bits): within 1e-5 of the terms' sizes.
 * Backward, f held constant (counts may be sums over several calls or
 * processes, and are then the whole batch's):
 *   grad_logits[t][e] = grad_losses[0]/N * p (f_e - sum_j f_j p_j)
 *       + grad_losses[1]/N * 2 lse p
 *       + sum over the token's routes k to e of
 *           topk_w[t][k] * (grad_topk_w[t][k] - sum_j topk_w[t][j] grad_topk_w[t][j])
 * The last line (the softmax over the selected logits that makes moe_route's
 * weights) only with topk_w and grad_topk_w, both or neither; without them
 * topk_ids may be NULL. Tokens that do not count get zeros.
 *   grad_losses [2] fp32, device.  grad_logits [T][E] fp32 out, 16-byte aligned.
 * n_experts <= 256, top_k <= min(8, n_experts), T < 2^28. workspace:
 * moe_balance_workspace_bytes (0 for few tokens: workspace may be NULL).
 */
size_t moe_balance_workspace_bytes(int32_t T, int32_t n_experts);
int moe_balance_loss(int32_t T, int32_t n_experts, int32_t top_k,
                     const float *logits, const int32_t *topk_ids,
                     const uint8_t *token_mask, int32_t *counts, float *losses,
                     void *workspace, size_t workspace_bytes, void *hip_stream);
int moe_balance_loss_backward(int32_t T, int32_t n_experts, int32_t top_k,
                              const float *logits, const int32_t *topk_ids,
                              const uint8_t *token_mask, const int32_t *counts,
                              const float *grad_losses, const float *topk_w,
                              const float *grad_topk_w, float *grad_logits,
                              void *hip_stream);

/*
 * 4-bit rows and their products (MXFP4, as the layer's expert weights are
 * stored): E2M1 codes, two per byte, the first in the low half, with one E8M0
 * scale byte (2^(b-127); 255: NaN) per 32 consecutive values of a row, for the
 * rows and the weights. They stand beside the layer's W4A16 projections, for
 * rows in 4 bits too (W4A4).
 *
 * Widths (cols, K) are multiples of 32 up to 65536, N up to 65536, rows below
 * 2^28. Codes and x 16-byte aligned, rows of x 16-byte aligned (pitches in
 * elements, at most 2^22; a pitch of codes in bytes); scales any address;
 * offsets, indices and out need the alignment of their type only. Zero rows
 * are a no-op.
 *
 * moe_fp4_quantize: x [rows][cols] (pitch ldx) of x_type to
 *   codes  [rows][cols/2]   e2m1(x / X), nearest, ties to even
 *   scales [rows][cols/32]  X = 2^max(e-2, -126), e the exponent of the group's
 *                           largest |x| rounded to two significant bits
 * so that |x / X| < 7 and every value is within half a step of E2M1. A group
 * that holds a NaN or an infinity gets scale 255 and codes 0: all of it NaN.
 * moe_fp4_swiglu: the same of h = silu(gate) * up in fp32; a row of gate_up
 * holds inter gate values, then inter up values.
 * moe_fp4_dequantize: codes and scales to out [rows][cols] (pitch ldo) of
 * out_type, exactly (past bf16's or fp32's range: infinite).
 */
int moe_fp4_quantize(int32_t rows, int32_t cols, const void *x, int64_t ldx,
                     int32_t x_type, uint8_t *codes, uint8_t *scales,
                     void *hip_stream);
int moe_fp4_swiglu(int32_t rows, int32_t inter, const void *gate_up, int64_t ld,
                   int32_t type, uint8_t *codes, uint8_t *scales,
                   void *hip_stream);
int moe_fp4_dequantize(int32_t rows, int32_t cols, const uint8_t *codes,
                       const uint8_t *scales, void *out, int64_t ldo,
                       int32_t out_type, void *hip_stream);

/* moe_fp4_linear: out[t][n] = sum over groups b of 32 of
 *     2^(x_scales[t][b] + w_scales[n][b] - 254) * sum_{k in b} x[t][k] * w[n][k]
 *   x [T][K] codes (pitch ldx bytes), x_scales [T][K/32],
 *   w [N][K] codes, w_scales [N][K/32],
 *   out [T][N] (pitch ldo) of out_type, rounded once from an fp32 sum. (A
 *   group's sum is exact; the order in which the groups are added goes by the
 *   sizes.)
 * moe_fp4_grouped: the same product for every expert over its own rows, with
 * moe_fp8_grouped's offsets, row_index, index_div and x_rows:
 *   x [x_rows][K], x_scales [x_rows][K/32], w [E][N][K], w_scales [E][N][K/32]
 *   (the layer's w13 and w2 as they are), out [rows][N].
 * n_experts <= 256; with row_index x_rows * ldx < 2^31. */
int moe_fp4_linear(int32_t T, int32_t N, int32_t K, const uint8_t *x,
                   int64_t ldx, const uint8_t *x_scales, const uint8_t *w,
                   const uint8_t *w_scales, void *out, int64_t ldo,
                   int32_t out_type, void *hip_stream);
int moe_fp4_grouped(int32_t rows, int32_t n_experts, int32_t N, int32_t K,
                    const int32_t *offsets, const int32_t *row_index,
                    int32_t index_div, int32_t x_rows, const uint8_t *x,
                    int64_t ldx, const uint8_t *x_scales, const uint8_t *w,
                    const uint8_t *w_scales, void *out, int64_t ldo,
                    int32_t out_type, void *hip_stream);

/*
 * The way into expert order and back, for rows of any router: what
 * moe_latent_forward does inside, as calls of their own, with gradients.
 *
 * moe_sort_routes: the routes r = t*K + k of topk_ids [T][K] int32, grouped by
 * expert. This process holds experts first_expert .. first_expert+n_experts-1;
 * routes to others (or to none: padding) are left out.
 *   expert_offsets [n_experts+1] int32 out: exclusive prefix sums of the
 *                    routes per expert; [n_experts]: routes that are here
 *   sorted_routes  [T*K] int32 out: route ids by expert, ascending within one;
 *                    behind the last: -1
 *   positions      [T][K] int32 out: where sorted_routes holds the route, or -1
 * workspace: moe_sort_workspace_bytes (0 for few routes: may be NULL).
 */
size_t moe_sort_workspace_bytes(int32_t T, int32_t n_experts, int32_t top_k);
int moe_sort_routes(int32_t T, int32_t n_experts, int32_t top_k,
                    const int32_t *topk_ids, int32_t first_expert,
                    int32_t *expert_offsets, int32_t *sorted_routes,
                    int32_t *positions, void *workspace, size_t workspace_bytes,
                    void *hip_stream);

/* moe_gather_rows: out[positions[t][k]] = x[t], x [T][cols] (pitch ldx), out
 * [rows][cols] (pitch ldo), both of type. Its gradient is moe_combine_rows of
 * the rows' gradients without weights.
 * moe_combine_rows: out[t] = sum_k topk_w[t][k] * x[positions[t][k]] in fp32,
 * k ascending, rounded once; x [rows][cols] (pitch ldx) of type, topk_w [T][K]
 * fp32 or NULL (all 1), out [T][cols] (pitch ldo) of out_type. A token with no
 * position gets zeros.
 * moe_combine_rows_backward, for grad_out [T][cols] (pitch ldg) of grad_type:
 *   grad_rows[positions[t][k]] = topk_w[t][k] * grad_out[t]   [rows][cols] of
 *                                type (pitch ldr), or NULL
 *   grad_w[t][k] = sum_c x[positions[t][k]][c] * grad_out[t][c]   [T][K] fp32,
 *                  or NULL (x is then not read and may be NULL); 0 for no position
 * Positions outside [0, rows) are none; no two may be the same row (that row
 * is then unspecified). n_taken: NULL, and rows that no position names are left
 * as they were; or a device int32 (moe_sort_routes' expert_offsets[n_experts]),
 * and rows from *n_taken on become zeros (no position may name one of them: that
 * row is then unspecified). Rows before it that no position names are left as
 * they were.
 * cols 1 .. 65536, top_k <= 8, T * top_k and rows below 2^28, pitches in
 * elements up to 2^22. Pointers need the alignment of their type only (rows of
 * a multiple of 8 values, all 16-byte aligned, are fastest). */
int moe_gather_rows(int32_t T, int32_t top_k, int32_t rows, int32_t cols,
                    const void *x, int64_t ldx, int32_t type,
                    const int32_t *positions, const int32_t *n_taken, void *out,
                    int64_t ldo, void *hip_stream);
int moe_combine_rows(int32_t T, int32_t top_k, int32_t rows, int32_t cols,
                     const void *x, int64_t ldx, int32_t type,
                     const int32_t *positions, const float *topk_w, void *out,
                     int64_t ldo, int32_t out_type, void *hip_stream);
int moe_combine_rows_backward(int32_t T, int32_t top_k, int32_t rows,
                              int32_t cols, const void *grad_out, int64_t ldg,
                              int32_t grad_type, const void *x, int64_t ldx,
                              int32_t type, const int32_t *positions,
                              const float *topk_w, const int32_t *n_taken,
                              void *grad_rows, int64_t ldr, float *grad_w,
                              void *hip_stream);

/* Their argument checks alone (callable without a GPU). */
int moe_fp8_quantize_validate(int32_t rows, int32_t cols, const void *x,
                              int64_t ldx, int32_t x_type, const uint8_t *codes,
                              const float *scales);
int moe_fp8_swiglu_validate(int32_t rows, int32_t inter, const void *gate_up,
                            int64_t ld, int32_t type, const uint8_t *codes,
                            const float *scales);
int moe_fp8_linear_validate(int32_t T, int32_t N, int32_t K, const uint8_t *x,
                            int64_t ldx, const float *x_scales, const uint8_t *w,
                            const float *w_scales, const void *out, int64_t ldo,
                            int32_t out_type);
int moe_fp8_grouped_validate(int32_t rows, int32_t n_experts, int32_t N,
                             int32_t K, const int32_t *offsets,
                             const int32_t *row_index, int32_t index_div,
                             int32_t x_rows, const uint8_t *x, int64_t ldx,
                             const float *x_scales, const uint8_t *w,
                             const float *w_scales, const void *out, int64_t ldo,
                             int32_t out_type);
int moe_balance_loss_validate(int32_t T, int32_t n_experts, int32_t top_k,
                              const float *logits, const int32_t *topk_ids,
                              const uint8_t *token_mask, const int32_t *counts,
                              const float *losses, const void *workspace,
                              size_t workspace_bytes);
int moe_balance_loss_backward_validate(int32_t T, int32_t n_experts,
                                       int32_t top_k, const float *logits,
                                       const int32_t *topk_ids,
                                       const uint8_t *token_mask,
                                       const int32_t *counts,
                                       const float *grad_losses,
                                       const float *topk_w,
                                       const float *grad_topk_w,
                                       const float *grad_logits);
int moe_fp4_quantize_validate(int32_t rows, int32_t cols, const void *x,
                              int64_t ldx, int32_t x_type, const uint8_t *codes,
                              const uint8_t *scales);
int moe_fp4_swiglu_validate(int32_t rows, int32_t inter, const void *gate_up,
                            int64_t ld, int32_t type, const uint8_t *codes,
                            const uint8_t *scales);
int moe_fp4_dequantize_validate(int32_t rows, int32_t cols, const uint8_t *codes,
                                const uint8_t *scales, const void *out,
                                int64_t ldo, int32_t out_type);
int moe_fp4_linear_validate(int32_t T, int32_t N, int32_t K, const uint8_t *x,
                            int64_t ldx, const uint8_t *x_scales,
                            const uint8_t *w, const uint8_t *w_scales,
                            const void *out, int64_t ldo, int32_t out_type);
int moe_fp4_grouped_validate(int32_t rows, int32_t n_experts, int32_t N,
                             int32_t K, const int32_t *offsets,
                             const int32_t *row_index, int32_t index_div,
                             int32_t x_rows, const uint8_t *x, int64_t ldx,
                             const uint8_t *x_scales, const uint8_t *w,
                             const uint8_t *w_scales, const void *out,
                             int64_t ldo, int32_t out_type);
int moe_sort_routes_validate(int32_t T, int32_t n_experts, int32_t top_k,
                             const int32_t *topk_ids, int32_t first_expert,
                             const int32_t *expert_offsets,
                             const int32_t *sorted_routes,
                             const int32_t *positions, const void *workspace,
                             size_t workspace_bytes);
int moe_gather_rows_validate(int32_t T, int32_t top_k, int32_t rows,
                             int32_t cols, const void *x, int64_t ldx,
                             int32_t type, const int32_t *positions,
                             const int32_t *n_taken, const void *out, int64_t ldo);
int moe_combine_rows_validate(int32_t T, int32_t top_k, int32_t rows,
                              int32_t cols, const void *x, int64_t ldx,
                              int32_t type, const int32_t *positions,
                              const float *topk_w, const void *out, int64_t ldo,
                              int32_t out_type);
int moe_combine_rows_backward_validate(
    int32_t T, int32_t top_k, int32_t rows, int32_t cols, const void *grad_out,
    int64_t ldg, int32_t grad_type, const void *x, int64_t ldx, int32_t type,
    const int32_t *positions, const float *topk_w, const int32_t *n_taken,
    const void *grad_rows, int64_t ldr, const float *grad_w);

/* Host-side evaluation of the tile orders of the prefill kernels (tests
 * check them over many shapes; no device work). For launch `kind`:
 *  MOE_TILES_DENSE  (0): the dense projection of an a x b output (pooler,
 *                         unpooler at prefill; b a multiple of its 256-column
 *                         tiles);
 *  MOE_TILES_EXPERT (1): the LDS-staged expert kernel over a row tiles (the
 *                         grid's bound) of b column tiles each;
 *  MOE_TILES_TILED  (2): the register-staged expert kernel, likewise.
 * Returns the launch's workgroup count G (or MOE_EINVAL for a bad kind or
 * size), and when out holds 2 * G ints writes (row tile, column tile) per
 * workgroup: (-1, -1) for a dense padding workgroup; row tiles of the expert
 * kernels beyond the tiles a call lists are skipped by the kernel itself. */
#define MOE_TILES_DENSE 0
#define MOE_TILES_EXPERT 1
#define MOE_TILES_TILED 2
int moe_tile_map(int32_t kind, int32_t a, int32_t b, int32_t *out, int32_t capacity);

/* Text of a status code (static storage). */
const char *moe_status_string(int status);

/* HIP error code of the last MOE_EHIP on the calling thread (0 if none). */
int moe_last_hip_error(void);

#ifdef __cplusplus
}
#endif

#endif /* MOE_H */

/*
 * moe.h - C ABI of the MI355X (gfx950) routed MoE block forward.
 *
 * The block, as the Olmo-core MoE report describes it ("Supercharging Olmo-core
 * for Efficient and Scalable MoE Training", Abstract; "Section 24: Conclusion",
 * 24.1 and Evidence 3 / Figure 74; explainer "Olmo-core 3: an open training
 * stack for trillion-parameter MoE", section "Olmo-core 3's answer: experts
 * resident, data routed"):
 *
 *   router logits -> softmax + top-k -> per-expert counts / offsets / positions
 *   computed and kept on the device -> rowwise dispatch that writes each token
 *   row straight into its expert's segment (no separate permutation) ->
 *   SwiGLU experts as a grouped GEMM whose group sizes never leave the device
 *   (no padding of experts to a common capacity) -> gate-weighted combine
 *   back to token order.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Pointers named as device pointers must point to device memory of the
 *    current HIP device; the caller owns every buffer.  The library never
 *    allocates device memory, never frees, never copies to the host and never
 *    synchronises inside these calls (except moe_kernel_times, the status
 *    query moe_fused_status and the comparison path moe_forward_host_sync,
 *    see there).
 *    All work is enqueued on `stream` (a hipStream_t; NULL = default stream),
 *    so calls on one stream are ordered and the whole sequence is capturable
 *    in a HIP graph.
 *  - Row-major layouts.  T tokens, d = d_model, E experts, k = top_k,
 *    H = d_hidden, R = T*k routed rows.
 *  - Storage types by `act_dtype`:
 *        MOE_F32   : x, xe, h, ye, y float32; weights float32.
 *        MOE_BF16  : x, xe, h, ye, y bfloat16; weights bfloat16; fp32 accumulate.
 *        MOE_MXFP8 : x bfloat16; xe and h are MXFP8 (E4M3 codes, one E8M0
 *                    scale byte per 32 consecutive elements along the GEMM
 *                    contraction axis); weights given bfloat16 and stored
 *                    MXFP8 by moe_pack_weights; ye and y bfloat16.
 *    Logits and gates are always float32; indices int32.
 *  - MXFP8 follows OCP Microscaling (MX) v1.0: E4M3 "FN" (bias 7, max 448, no
 *    infinities), shared exponent floor(log2(amax)) - 8 clamped to [-127,127]
 *    (all-zero block -> 2^-127), elements rounded to nearest-even, saturated
 *    to +-448, sign kept on zero.  Payload 33/32 bytes per value (report
 *    Section 24, Evidence 10).
 *  - Routing: experts ranked by float32 logit, ties to the lower expert index
 *    (-0.0 == +0.0); slot j of a token holds its j-th largest logit.  Gates
 *    are the softmax over all E renormalised over the k selected experts.
 *    Rows of one expert are ordered by ascending token index (stable), experts
 *    back to back without padding: offsets[e] = sum of counts[e' < e].
 *  - Shapes supported: 1 <= k <= min(E, 16), E <= 1024, T >= 1, and
 *    d, H multiples of 64 (MOE_F32, MOE_BF16) or of 128 (MOE_MXFP8); the
 *    bytes of an [R, max(d, H)] activation buffer and of one expert's
 *    [2H, d] weights must each stay below 2^32.
 *  - Errors: every entry point returns MOE_OK or a negative MOE_ERR_* code.
 *    Arguments are validated on the host before anything is enqueued; a
 *    failed check enqueues nothing.  MOE_ERR_LAUNCH reports hipGetLastError()
 *    after a launch.  Faults inside kernels surface at the caller's next
 *    synchronisation.  Preconditions not checked: logits are finite; pos /
 *    offsets buffers come from moe_route for the same problem.
 */
#ifndef MOE_MI355X_H
#define MOE_MI355X_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_OK             0
#define MOE_ERR_NULL      -1   /* a required pointer is NULL                      */
#define MOE_ERR_SHAPE     -2   /* unsupported T, d, E, k or H                      */
#define MOE_ERR_DTYPE     -3   /* unknown act_dtype, or flag not valid for it      */
#define MOE_ERR_WORKSPACE -4   /* ws_bytes smaller than moe_workspace_bytes()      */
#define MOE_ERR_LAUNCH    -5   /* a kernel launch or HIP runtime call failed       */
#define MOE_ERR_STATE     -6   /* no profiled forward yet; inconsistent host counts */
#define MOE_ERR_ARG       -7   /* a setting outside its documented range, or a
                                * pointer not aligned or not distinct as documented */

#define MOE_F32   0
#define MOE_BF16  1
#define MOE_MXFP8 2

/* flags */
#define MOE_LOGITS_GIVEN     1  /* logits are an input; skip the router GEMM x . W_r     */
#define MOE_IDENTITY_EXPERTS 2  /* test mode of moe_forward: ye := xe (f32 / bf16 only)  */
/* MOE_KEEP_GATE_UP: moe_forward also stores the experts' pre-activations
 * a | b = xe W1 (bf16 of GEMM1's float32 accumulators, [T*k][2H] in the
 * packed column order) in its workspace, and moe_backward reads them instead
 * of recomputing xe W1.  The report treats recompute as an option that trades
 * throughput for activation memory ("Section 24: Conclusion", Evidence 11;
 * its per-block recompute cost about a fifth of the throughput); without this
 * flag the library recomputes, with it the forward keeps 4 T k H more bytes.
 * MOE_BF16 (d_model, d_hidden >= 128: the fused FFN's blocks): the gradients
 * are bit for bit those of the recomputing path.  MOE_MXFP8: the stored a | b
 * come from the forward's MXFP8 GEMM, the recompute is a bf16 GEMM of the
 * dequantised values, so the gradients differ by their accumulation order
 * only.  Any other problem with the flag is MOE_ERR_DTYPE.  moe_forward and
 * moe_forward_host_sync honour it; the staged calls ignore it.  moe_backward
 * must be given the problem (flags included) its moe_forward ran with: with
 * the flag it reads a | b from fwd_ws, whose size then includes them (a
 * forward workspace sized without the flag is MOE_ERR_WORKSPACE). */
#define MOE_KEEP_GATE_UP     4

typedef struct moe_problem {
    int32_t T;          /* tokens                                 */
    int32_t d_model;    /* d                                      */
    int32_t n_experts;  /* E                                      */
    int32_t top_k;      /* k                                      */
    int32_t d_hidden;   /* H, expert SwiGLU hidden size           */
    int32_t act_dtype;  /* MOE_F32 | MOE_BF16 | MOE_MXFP8         */
    int32_t flags;      /* MOE_LOGITS_GIVEN | MOE_IDENTITY_EXPERTS | MOE_KEEP_GATE_UP */
} moe_problem;

/* Library version string and a readable name of a status code (host only). */
const char* moe_version(void);
const char* moe_status_string(int32_t status);

/* Device workspace, in bytes, that is enough for every entry point below on
 * problem p (host only, no GPU call).  Contents need no initialisation and are
 * overwritten by every call.  The caller allocates it once and passes it to
 * every call, so the block's buffers keep fixed addresses from step to step
 * (report "Section 24: Conclusion", 24.3: graph replay needs buffers at stable
 * addresses, reused only after their last consumer).  Errors: MOE_ERR_NULL,
 * MOE_ERR_SHAPE / MOE_ERR_DTYPE for an invalid problem. */
int32_t moe_workspace_bytes(const moe_problem* p, size_t* bytes);

/* Size in bytes of the packed expert weights for p (host only, no GPU call):
 * the regions moe_pack_weights writes, described there (report "Section 24:
 * Conclusion", 24.3: weight caches built once, in the layout the GEMM reads).
 * Errors: as moe_workspace_bytes. */
int32_t moe_packed_weight_bytes(const moe_problem* p, size_t* bytes);

/* Packs the expert weights once, outside the timed path: re-lays them out with
 * the contraction axis contiguous and, for MOE_MXFP8, quantises them (report
 * "Section 24: Conclusion", 24.3: MXFP8 weight caches kept beside the
 * high-precision weights, produced by a quantiser in the layout the GEMM
 * consumes, so no per-step conversion kernel runs).  The caller owns both
 * buffers; the inputs are not modified.  Errors: MOE_ERR_NULL for a NULL
 * pointer, shape/dtype errors as moe_workspace_bytes; nothing is enqueued on
 * an error.
 *   w_gate, w_up : device [E, d, H]   (x . W convention), storage type above
 *   w_down       : device [E, H, d]
 *   packed       : device, moe_packed_weight_bytes() bytes, layout:
 *     W1 [E][2H][d] : row n of expert e is gate column h = 32*(n/64) + n%32 when
 *                     (n/32) is even, else up column h (same formula); i.e. 32
 *                     gate columns then the matching 32 up columns, repeated.
 *     W2 [E][d][H]  : W2[e][n][j] = w_down[e][j][n].
 *     Elements are float32 / bfloat16 / E4M3 by act_dtype.  For MOE_MXFP8 the
 *     E8M0 scales follow, each covering 32 consecutive elements of a row and
 *     stored slice-major: S1 [E][d/128][2H][4], then S2 [E][H/128][d][4], where
 *     S[e][s][n][j] is the scale of elements [128 s + 32 j, 128 s + 32 j + 32)
 *     of packed row n (the layout the GEMM loads without conversion).
 *   Regions are W1, W2, S1, S2 in that order, each starting at a multiple of
 *   256 bytes. */
int32_t moe_pack_weights(const moe_problem* p, const void* w_gate, const void* w_up,
                         const void* w_down, void* packed, void* stream);

/* Routing (report: count routes on the GPU, metadata kept on the device,
 * Section 24.1 and Evidence 3).
 *   x        : device [T, d] (storage type of act_dtype; MXFP8: bfloat16);
 *              unused (may be NULL) with MOE_LOGITS_GIVEN
 *   w_router : device [d, E], same type as x; unused with MOE_LOGITS_GIVEN
 *   logits   : device float32 [T, E]; input with MOE_LOGITS_GIVEN, else output
 *   topk_idx : device int32 [T, k] out;  topk_gate : device float32 [T, k] out
 *   counts   : device int32 [E] out;     offsets   : device int32 [E+1] out
 *   pos      : device int32 [T, k] out, row of (token, slot) in the expert-major
 *              buffer: offsets[e] + number of earlier tokens routed to e
 *   row_token: device int32 [R] out, row_token[pos[t][j]] = t
 *   router_stats : device float32 [E + 2] out, or NULL to skip.  The report
 *              asks that the requested route counts be inspected next to the
 *              Switch-style balance scalar, which mixes soft router scores with
 *              hard counts ("Section 24: Conclusion", 24.3 and Evidence 9 /
 *              Figure 45); its formula is not printed, the Switch form is used:
 *                [e]     P_e = mean over tokens of softmax(logits[t])[e]
 *                [E]     E * sum_e (counts[e] / (T k)) * P_e
 *                [E + 1] max_e counts[e] / (T k / E)   (worst-case load / mean)
 *              Computed in the top-k pass; sums run in a fixed order, so the
 *              values are reproducible bit for bit.
 *   ws       : device workspace of ws_bytes bytes */
int32_t moe_route(const moe_problem* p, const void* x, const void* w_router, float* logits,
                  int32_t* topk_idx, float* topk_gate, int32_t* counts, int32_t* offsets,
                  int32_t* pos, int32_t* row_token, float* router_stats, void* ws, size_t ws_bytes,
                  void* stream);

/* moe_route for callers that cannot allocate device memory: code under HIP
 * graph capture, tight serving loops, and harnesses that forbid hipMalloc.
 * Arguments, outputs and results are those of moe_route (bit for bit: the
 * same kernels run); there is no workspace argument.  The routing scratch
 * (per-block expert histograms and bases, per-block router-probability
 * partials and, for a bfloat16 / MXFP8 learned router, the transposed router
 * weights) lives in a library-owned device array of MOE_ROUTE_SCRATCH_BYTES
 * bytes, one per GPU, set up on the first call on that GPU and held until
 * the process ends.  The call allocates and frees nothing.
 * The kernels write every scratch byte they read, so no state carries from
 * one call to the next; but every call on one GPU uses that GPU's single
 * array, so calls that overlap on one GPU (other streams, other threads)
 * race and give wrong results: serialise them.
 * Errors: as moe_route; MOE_ERR_WORKSPACE (nothing enqueued) when the
 * problem's routing scratch, the routing part of moe_workspace_bytes' layout
 * (about ceil(T/256) * E * (12 + 4 G) bytes, G <= 64 the lanes per token in
 * top-k selection, plus E * d * 2 for a bfloat16 / MXFP8 learned router,
 * each region rounded up to 256 bytes), exceeds MOE_ROUTE_SCRATCH_BYTES;
 * MOE_ERR_LAUNCH if the array's device address cannot be obtained. */
#define MOE_ROUTE_SCRATCH_BYTES (4 << 20)
int32_t moe_route_noalloc(const moe_problem* p, const void* x, const void* w_router, float* logits,
                          int32_t* topk_idx, float* topk_gate, int32_t* counts, int32_t* offsets,
                          int32_t* pos, int32_t* row_token, float* router_stats, void* stream);

/* Rowwise dispatch (report Abstract: each token row written directly into its
 * expert's buffer): xe[pos[t][j]] = x[t] for every slot.
 *   x        : device [T, d]
 *   pos      : device int32 [T, k] from moe_route
 *   xe       : device [R, d] out (MOE_MXFP8: uint8 E4M3 codes), 16-byte aligned
 *   xe_scale : device uint8 [d/128][R][4], 4-byte aligned, out for MOE_MXFP8, else ignored (may
 *              be NULL): xe_scale[s][r][j] is the E8M0 scale of elements
 *              [128 s + 32 j, 128 s + 32 j + 32) of row r, so the four scales
 *              of a 128-wide slice of a row form one dword and the dwords of
 *              consecutive rows are adjacent, the layout the grouped GEMM reads
 *              directly (report "Section 24: Conclusion", 24.3: a quantiser
 *              should emit what the consumer reads without conversion) */
int32_t moe_dispatch(const moe_problem* p, const void* x, const int32_t* pos, void* xe,
                     uint8_t* xe_scale, void* stream);

/* Expert SwiGLU FFN as a grouped GEMM whose groups are read from device
 * memory (report: device-scheduled grouped GEMM, no padding to a capacity):
 *   for every expert e and row r in [offsets[e], offsets[e+1]):
 *     h  = silu(xe[r] . W_gate[e]) * (xe[r] . W_up[e])   (stored in workspace)
 *     ye[r] = h . W_down[e]
 *   xe, xe_scale : as written by moe_dispatch
 *   packed_w     : from moe_pack_weights
 *   offsets      : device int32 [E+1] from moe_route
 *   ye           : device [R, d] out (float32 for MOE_F32, else bfloat16)
 *   ws           : workspace (holds h and, for bfloat16, the counters of the
 *                  fused launch, cleared by each call; calls sharing a
 *                  workspace must not overlap)
 * bfloat16 (d_model and d_hidden >= 128) runs both projections in one
 * persistent launch: a GEMM2 tile starts once the GEMM1 tiles of its rows have
 * finished, so neither GEMM ends in a partly filled round.  That wait is
 * bounded (about 2 s) so that the launch cannot hang the GPU: if other work
 * kept this launch's GEMM1 workgroups off the compute units for longer, the
 * GEMM2 tile stops waiting, writes its rows of ye as NaN (never a wrong
 * finite value) and sets an error word in the workspace, which
 * moe_fused_status reports.  The grid never exceeds the device's compute-unit
 * count, so on an otherwise idle GPU every wait ends normally.
 * Every output tile is computed whole by one workgroup in a fixed K order, so
 * the result does not depend on the grid (moe_set_gemm_grid_cap). */
int32_t moe_grouped_swiglu(const moe_problem* p, const void* xe, const uint8_t* xe_scale,
                           const void* packed_w, const int32_t* offsets, void* ye, void* ws,
                           size_t ws_bytes, void* stream);

/* Combine back to token order (report Abstract: combine without a permutation):
 *   y[t] = sum over j = 0..k-1, in slot order, of topk_gate[t][j] * ye[pos[t][j]],
 *   accumulated in float32 and rounded to nearest-even into y.
 *   ye : device [R, d]; y : device [T, d] out (float32 for MOE_F32, else bfloat16) */
int32_t moe_combine(const moe_problem* p, const void* ye, const float* topk_gate,
                    const int32_t* pos, void* y, void* stream);

/* The whole block on one stream: route, dispatch, grouped SwiGLU, combine, with
 * no host synchronisation between them.  For MOE_BF16 with d_model and
 * d_hidden >= 128 the dispatch is not materialised: the fused grouped GEMM
 * reads each expert-major row r straight from x[row_token[r]] (the row the
 * dispatch would have copied), so no xe is written and the routing pass only
 * finalises pos and row_token.  For MOE_MXFP8 with d_model >= 256 each token
 * row is quantised once (codes and scales per token, not per routed row),
 * GEMM1 reads the code rows through row_token, and only the E8M0 scales are
 * laid out per expert-major row.  y is the same either way ("Supercharging Olmo-core ...",
 * Section 2, the design paragraph after Figure 5: no extra permutation, no
 * device-to-host synchronisation and no gap between launches; Abstract:
 * device-scheduled grouped GEMMs).  The caller owns every buffer; ws is at
 * least moe_workspace_bytes(p) bytes, and calls sharing a workspace must not
 * overlap.  All arguments are validated on the host before anything is
 * enqueued: a non-zero status means nothing ran.  Arguments as above; topk_idx,
 * topk_gate, counts, offsets, pos and router_stats are optional outputs (NULL:
 * kept in the workspace only, or for router_stats not computed).  With
 * MOE_IDENTITY_EXPERTS the grouped GEMM is skipped and ye := xe (MOE_F32 /
 * MOE_BF16 only), so y[t] = x[t] * sum_j gate[t][j]. */
int32_t moe_forward(const moe_problem* p, const void* x, const void* w_router, float* logits,
                    const void* packed_w, void* y, int32_t* topk_idx, float* topk_gate,
                    int32_t* counts, int32_t* offsets, int32_t* pos, float* router_stats, void* ws,
                    size_t ws_bytes, void* stream);

/* The same block with one host wait, for comparison with moe_forward: the
 * original MoE path the report measures against needed the per-expert routing
 * counts on the CPU before the grouped-GEMM group sizes were known ("Section
 * 24: Conclusion", 24.1 and Evidence 3 / Figure 74: one device-to-host copy
 * and host wait per routed block).  After routing, the counts are copied to
 * host_counts (host memory of E int32, owned by the caller; pinned memory
 * avoids a staging copy) and the calling thread waits for the stream before it
 * sizes the grouped-GEMM grids from them and enqueues the rest.  Every output
 * is bit-identical to moe_forward's (same kernels; only the grid size and the
 * wait differ).  Not capturable in a HIP graph.  With profiling on (below) the
 * stage "host_count_wait" is the GPU time from the end of routing until work
 * resumes after the wait.  Errors: as moe_forward, MOE_ERR_NULL for a NULL
 * host_counts, MOE_ERR_STATE if the copied counts do not sum to T*k. */
int32_t moe_forward_host_sync(const moe_problem* p, const void* x, const void* w_router, float* logits,
                              const void* packed_w, void* y, int32_t* topk_idx, float* topk_gate,
                              int32_t* counts, int32_t* offsets, int32_t* pos, float* router_stats, void* ws,
                              size_t ws_bytes, void* stream, int32_t* host_counts);

/* Per-kernel timing of moe_forward with HIP events recorded on its stream.
 * moe_set_profiling(1) makes later moe_forward calls record an event before
 * the first kernel and after each kernel (events are created on first use and
 * kept; the last 128 calls keep separate events).  moe_set_profiling resets
 * the count of profiled calls.  moe_kernel_times waits for the last profiled
 * call to finish (this call synchronises on its final event) and writes up to
 * max_n stage names and their durations in milliseconds averaged over the
 * profiled calls (at most the last 128); *n receives the number of stages.
 * Returns MOE_ERR_STATE when no profiled call completed its launches.  Not for
 * use while a graph capture of moe_forward is in progress. */
int32_t moe_set_profiling(int32_t enable);

int32_t moe_kernel_times(const char** names, float* ms, int32_t max_n, int32_t* n);

/* Caps the persistent grid of the bf16 and MXFP8 grouped GEMMs at `cap`
 * workgroups (one per compute unit; a multiple of 8 in [8, 256]), for callers
 * that keep compute units free for concurrent work on another stream; 0
 * removes the cap.  Process-wide, applies to calls launched afterwards; not
 * for use while another thread launches.  Returns MOE_ERR_ARG for any other
 * value. */
int32_t moe_set_gemm_grid_cap(int32_t cap);

/* Test hooks for the fused bfloat16 grouped GEMMs (the forward expert FFN of
 * moe_grouped_swiglu / moe_forward and the backward's data-gradient chain):
 * MOE_TEST_FFN_WAIT makes every dependent tile skip the early check of its
 * rows and start only after waiting for them (the path a tile takes when its
 * rows are not yet done), so tests can show that this path gives the same
 * result; outputs are unchanged, only speed drops.  MOE_TEST_FFN_GIVE_UP makes
 * every such wait end at once as if its bound had been reached, without
 * looking at the counter: the tile writes NaN and raises the error word that
 * moe_fused_status reports (every kernel still runs to completion), so tests
 * can check the failure path.  Process-wide, applies to calls launched
 * afterwards; 0 clears them.  Returns MOE_ERR_ARG for unknown bits. */
#define MOE_TEST_FFN_WAIT 1
#define MOE_TEST_FFN_GIVE_UP 2
int32_t moe_set_test_flags(int32_t flags);

/* Outcome of the bounded dependency waits of the last fused grouped-GEMM
 * launch that used workspace ws (the report's Section 24.3 asks that buffers be
 * reused only after their last consumer has finished and that such
 * dependencies be explicit at component interfaces; in the fused launches one
 * GEMM's tiles consume rows another GEMM's tiles produce, and a tile that
 * stops waiting for its producers makes the broken dependency explicit here).
 *   which  : MOE_STATUS_FORWARD for the workspace of moe_forward /
 *            moe_forward_host_sync / moe_grouped_swiglu (ws_bytes >= the
 *            grouped-GEMM part of moe_workspace_bytes), MOE_STATUS_BACKWARD
 *            for the workspace of moe_backward (ws_bytes >=
 *            moe_backward_workspace_bytes)
 *   status : host int32 out: MOE_OK, or MOE_ERR_STATE if some dependent tile
 *            gave up waiting, in which case its output rows (ye in the
 *            forward; dh, da | db or dxe and what derives from them in the
 *            backward) hold NaN.
 * The word is cleared by every call that launches a fused kernel on ws, so it
 * describes the last such call; for problems that run no fused launch (other
 * dtypes or small d, H) the status is MOE_OK without a device access.
 * Synchronises: the word is copied to the host after the work already queued
 * on `stream` and the calling thread waits for it. */
#define MOE_STATUS_FORWARD 0
#define MOE_STATUS_BACKWARD 1
int32_t moe_fused_status(const moe_problem* p, const void* ws, size_t ws_bytes, int32_t which, int32_t* status,
                         void* stream);

/* ---------------------------------------------------------------- backward
 *
 * Gradients of the block for a loss L with dL/dy = dy (MOE_IDENTITY_EXPERTS
 * returns MOE_ERR_DTYPE).  The report runs the block's backward with the
 * dispatch and combine as each other's transposes, grouped GEMMs for data and
 * weight gradients and the block forward re-executed ("Section 24:
 * Conclusion", Evidence 7 and Evidence 11).  With g the gates (the softmax of
 * the k selected logits):
 *
 *   dgate[t,j] = dy[t] . ye[pos[t,j]]          dye[pos[t,j]] = g[t,j] dy[t]
 *   dlogits[t,e_j] = g_j (dgate_j - sum_i g_i dgate_i), 0 for unselected e
 *   a | b = xe W1 (recomputed, or stored with MOE_KEEP_GATE_UP);  dh = dye W_down^T
 *   da = dh b silu'(a);  db = dh silu(a);  dxe = da W_gate^T + db W_up^T
 *   dw_down[e] = h^T dye,  dw_gate[e] = xe^T da,  dw_up[e] = xe^T db
 *                                              (sums over expert e's rows)
 *   dx[t] = sum_j dxe[pos[t,j]]  (+ dlogits[t] W_r^T for the learned router)
 *   dw_router = x^T dlogits                     (learned router only; summed
 *               per expert over that expert's token rows)
 *
 * Storage: dye, a, b, dh, da, db, dxe and dx in the activation type (bf16
 * rounded to nearest even where stored), dlogits and all weight gradients
 * float32.  MOE_MXFP8 blocks follow Evidence 7 (dequantise, then bf16): the
 * saved MXFP8 xe and h are dequantised to bf16 (exactly), the weights are the
 * bf16 values of the forward's MXFP8 weights, and every step above runs in
 * bf16 (dy, dx bf16).  Every reduction runs in a fixed order: results are
 * bitwise reproducible.  All work is enqueued on `stream`; nothing allocates
 * or synchronises, so the call is capturable in a HIP graph.
 *
 * moe_backward_weight_bytes / moe_pack_weights_backward: the backward weight
 * cache (the report's second weight cache, 24.3), built once from w_gate,
 * w_up [E, d, H] and w_down [E, H, d] (device, the activation type; bf16 for
 * MOE_MXFP8): W1T [E][d][2H], row c holding for each column n of the packed
 * W1 (32 gate then 32 up hidden units per 64) the weight of input c; W_down
 * [E][H][d]; for MOE_MXFP8 also the packed W1 in bf16.  MOE_MXFP8 stores the
 * dequantised MXFP8 values (blocks of 32 along each forward GEMM's
 * contraction axis, as moe_pack_weights quantises them).
 *
 * moe_backward arguments (device pointers unless noted):
 *   dy          [T, d] activation type (bf16 for MOE_MXFP8)
 *   x           [T, d] the forward's input.  Required for the learned router
 *               and for MOE_BF16 blocks with d_model and d_hidden >= 128 (their
 *               forward reads the token rows in place and keeps no dispatched
 *               copy, so the backward gathers them from x again); otherwise
 *               unused and may be NULL
 *   w_router    [d, E] activation type (learned router only; may be NULL with
 *               MOE_LOGITS_GIVEN)
 *   packed_w    the forward weight cache (moe_pack_weights); unused, may be
 *               NULL, for MOE_MXFP8
 *   packed_bwd  the backward weight cache (moe_pack_weights_backward)
 *   topk_idx, topk_gate, offsets, pos : the forward's routing arrays, or NULL
 *               for the copies moe_forward kept in its workspace when it was
 *               given NULL for them
 *   fwd_ws      the workspace of the moe_forward call being differentiated,
 *               unchanged since (it holds h, ye, row_token and the dispatched
 *               rows: none for the gathering bf16 blocks above, one MXFP8
 *               code row per token for MXFP8 blocks with d_model >= 256, one
 *               per routed row otherwise; with MOE_KEEP_GATE_UP also a | b);
 *               fwd_ws_bytes >= moe_workspace_bytes
 *   dx          [T, d] out, activation type (bf16 for MOE_MXFP8)
 *   dlogits     [T, E] out, float32
 *   dw_gate, dw_up [E, d, H] out, dw_down [E, H, d] out, float32
 *   dw_router   [d, E] out, float32 (learned router only; may be NULL with
 *               MOE_LOGITS_GIVEN)
 *   ws          backward workspace, ws_bytes >= moe_backward_workspace_bytes
 * Errors: as moe_forward; MOE_ERR_SHAPE also when T*k*2H elements of the
 * backward's activation type exceed 2^32 bytes. */
int32_t moe_backward_workspace_bytes(const moe_problem* p, size_t* bytes);
int32_t moe_backward_weight_bytes(const moe_problem* p, size_t* bytes);
int32_t moe_pack_weights_backward(const moe_problem* p, const void* w_gate, const void* w_up, const void* w_down,
                                  void* packed_bwd, void* stream);
int32_t moe_backward(const moe_problem* p, const void* dy, const void* x, const void* w_router, const void* packed_w,
                     const void* packed_bwd, const int32_t* topk_idx, const float* topk_gate, const int32_t* offsets,
                     const int32_t* pos, const void* fwd_ws, size_t fwd_ws_bytes, void* dx, float* dlogits,
                     float* dw_gate, float* dw_up, float* dw_down, float* dw_router, void* ws, size_t ws_bytes,
                     void* stream);

/* ---------------------------------------------------------------- the norm in front of the block
 *
 * Root-mean-square norm with the residual's addition, per token row:
 *   s[t] = x[t] + residual[t],  rstd[t] = (mean_c s[t][c]^2 + eps)^(-1/2),
 *   y[t][c] = s[t][c] rstd[t] weight[c]
 * with s the float32 sum and its squares summed in float64; sum and y are
 * rounded to nearest even where they are stored (y from the float32 s), for
 * rows of any finite sums
 * (rstd itself is infinite past float32's range).  For MOE_MXFP8 problems the
 * rows' MXFP8 form can be written in the same pass: E4M3 codes and E8M0 scales
 * of the stored bf16 y (MXFP8 as above, blocks of 32 along d; NaN saturated, as
 * moe_forward's own quantiser does), which moe_forward_quantized reads
 * ("Section 24: Conclusion", 24.3: a quantiser should emit what the consumer
 * reads without conversion; Evidence 6 counted separate quantise kernels as
 * overhead).  Uses T, d_model and act_dtype of the problem.
 *   x        : device [T, d] activation type (bf16 for MOE_MXFP8)
 *   residual : device [T, d], or NULL: s = x
 *   weight   : device [d], activation type
 *   eps      : finite, >= 0
 *   sum      : device [T, d] out, or NULL; may be x or residual (in place)
 *   y        : device [T, d] out, may be x or residual (in place, if sum is
 *              not the same); NULL only with yq
 *   yq       : device uint8 [T, d] out, MOE_MXFP8 only, or NULL
 *   yq_scale : device uint8 [T, d/32] out with yq, 4-byte aligned
 *   rstd     : device float32 [T] out, or NULL (moe_norm_backward reads it)
 * Tensors [T, d] and weight are 16-byte aligned, yq 8-byte aligned.
 * Errors: MOE_ERR_NULL (x, weight, y and yq both, yq without yq_scale),
 * MOE_ERR_DTYPE for yq on another act_dtype, MOE_ERR_ARG for eps, an
 * unaligned pointer or y == sum. */
int32_t moe_norm(const moe_problem* p, const void* x, const void* residual, const void* weight, float eps, void* sum,
                 void* y, uint8_t* yq, uint8_t* yq_scale, float* rstd, void* stream);

/* Gradients of moe_norm: with n = s rstd and u = dy weight,
 *   ds[t] = rstd (u - n mean_c(u n)) + dsum[t],   dweight = sum_t dy n.
 * ds is the gradient of x and of the residual alike.
 *   dy      : device [T, d] activation type, the gradient of y
 *   dsum    : device [T, d], the gradient of sum from its other consumers (the
 *             residual stream), or NULL
 *   s       : device [T, d], the forward's sum (x without a residual)
 *   rstd    : device float32 [T] of the forward
 *   ds      : device [T, d] out, may be dy or dsum (in place)
 *   dweight : device float32 [d] out
 *   ws      : device, moe_norm_backward_workspace_bytes (host-only query);
 *             calls sharing a workspace must not overlap, here and below
 * Sums run in a fixed order (bitwise reproducible).  Tensors 16-byte aligned
 * (rstd 4).  Errors: MOE_ERR_NULL, MOE_ERR_WORKSPACE, MOE_ERR_ARG for an
 * unaligned pointer or ds == s. */
int32_t moe_norm_backward_workspace_bytes(const moe_problem* p, size_t* bytes);
int32_t moe_norm_backward(const moe_problem* p, const void* dy, const void* dsum, const void* s, const void* weight,
                          const float* rstd, void* ds, float* dweight, void* ws, size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------- layer norm in front of the block
 *
 * Layer norm with the residual's addition, for models that subtract a row's mean:
 *   s[t] = x[t] + residual[t],  mean[t] = mean_c s[t][c],
 *   rstd[t] = (mean_c (s[t][c] - mean[t])^2 + eps)^(-1/2),
 *   y[t][c] = (s[t][c] - mean[t]) rstd[t] weight[c] + bias[c]
 * with s the float32 sum, the means and y taken in float64 from it and rounded to
 * nearest even where they are stored.  A row of one value everywhere gives the
 * bias (eps > 0; with eps 0 it is NaN).  MXFP8 codes of the stored y, layouts,
 * optional arguments and buffers that may be the same are moe_norm's.
 *   weight   : device [d], activation type
 *   bias     : device [d], activation type, or NULL: none
 *   mean     : device float32 [T] out, or NULL (moe_layer_norm_backward reads it)
 * Errors: as moe_norm, with bias and mean among the pointers. */
int32_t moe_layer_norm(const moe_problem* p, const void* x, const void* residual, const void* weight, const void* bias,
                       float eps, void* sum, void* y, uint8_t* yq, uint8_t* yq_scale, float* mean, float* rstd,
                       void* stream);

/* Gradients of moe_layer_norm: with n = (s - mean) rstd and u = dy weight,
 *   ds[t] = rstd (u - mean_c(u) - n mean_c(u n)) + dsum[t],
 *   dweight = sum_t dy n,  dbias = sum_t dy.
 *   mean, rstd     : device float32 [T] of the forward
 *   dweight, dbias : device float32 [d] out; dbias may be NULL
 * Other arguments, in-place use, order of the sums and errors as
 * moe_norm_backward; ws: moe_layer_norm_backward_workspace_bytes. */
int32_t moe_layer_norm_backward_workspace_bytes(const moe_problem* p, size_t* bytes);
int32_t moe_layer_norm_backward(const moe_problem* p, const void* dy, const void* dsum, const void* s,
                                const void* weight, const float* mean, const float* rstd, void* ds, float* dweight,
                                float* dbias, void* ws, size_t ws_bytes, void* stream);

/* moe_forward of a MOE_MXFP8 block (d_model >= 256) whose token rows are
 * already quantised: xq [T, d] codes and xq_scale [T, d/32] as moe_norm
 * writes them (xq 16-byte, xq_scale 4-byte aligned).  No quantise pass runs;
 * GEMM1 reads the given code rows.  x (bf16) is read by the learned router
 * only and may be NULL with MOE_LOGITS_GIVEN.  Every output is bit for bit
 * moe_forward's of the rows the codes were made from.  The codes are not
 * copied to the workspace: a backward of this call is moe_backward_aux with
 * the same xq.  Errors: as moe_forward, MOE_ERR_DTYPE for another act_dtype,
 * MOE_ERR_SHAPE for d_model < 256, MOE_ERR_ARG for an unaligned pointer. */
int32_t moe_forward_quantized(const moe_problem* p, const void* x, const uint8_t* xq, const uint8_t* xq_scale,
                              const void* w_router, float* logits, const void* packed_w, void* y, int32_t* topk_idx,
                              float* topk_gate, int32_t* counts, int32_t* offsets, int32_t* pos, float* router_stats,
                              void* ws, size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------- the router's losses
 *
 * Balance and z loss of the router with the per-expert counts (the report
 * asks that requested counts be inspected next to the Switch-style scalar,
 * "Section 24: Conclusion", 24.3 and Evidence 9 / Figure 45).  Over the N live
 * tokens, p_t the softmax of logits[t], f_e = counts[e] / (N k):
 *   loss[0] = E sum_e f_e P_e,  P_e = (1/N) sum_t p_te
 *   loss[1] = (1/N) sum_t lse_t^2,  lse_t = log sum_e exp logits[t][e]
 * moe_balance_loss_backward: with dloss = (g0, g1) and the counts constants,
 *   dlogits[t][e] = (p_te / N) (g0 E (f_e - sum_j f_j p_tj) + 2 g1 lse_t),
 * zero for tokens that are not live.  N = 0 gives zeros.  Uses T, n_experts
 * and top_k of the problem.
 *   logits : device float32 [T, E]; -inf excludes an expert from the softmax,
 *            a live row of -inf alone counts as p = 0, lse = 0; NaN in a live
 *            row makes both losses and that row's gradient NaN; rows that are
 *            not live may hold anything
 *   topk_idx : device int32 [T, k]; an index outside [0, E) is not counted
 *   mask   : device uint8 [T], nonzero: the token is live; NULL: all are
 *   counts : device int32 [E + 1]: out / in; counts[E] is N
 *   loss   : device float32 [2] out
 *   dloss  : device float32 [2], the gradient for the two losses
 *   dlogits: device float32 [T, E] out
 *   ws     : device, moe_balance_workspace_bytes (host-only query)
 * dlogits may be logits (in place).  logits, dlogits and ws are 16-byte
 * aligned.  Sums run in a fixed order (bitwise reproducible).  Errors:
 * MOE_ERR_NULL, MOE_ERR_WORKSPACE, MOE_ERR_ARG for an unaligned pointer. */
int32_t moe_balance_workspace_bytes(const moe_problem* p, size_t* bytes);
int32_t moe_balance_loss(const moe_problem* p, const float* logits, const int32_t* topk_idx, const uint8_t* mask,
                         int32_t* counts, float* loss, void* ws, size_t ws_bytes, void* stream);
int32_t moe_balance_loss_backward(const moe_problem* p, const float* logits, const uint8_t* mask,
                                  const int32_t* counts, const float* dloss, float* dlogits, void* stream);

/* Gradients of the router's product logits = x W_r from dense logit gradients:
 *   dx[t] = dx_in[t] + sum_e dlogits[t][e] W_r[:, e],   dw_router = x^T dlogits
 * accumulated in float32 (float32 operands enter the matrix cores as three
 * bfloat16 terms each), dx rounded once.  Infinite and NaN operands give what
 * the sums of products give.
 *   dlogits  : device float32 [T, E]
 *   x        : device [T, d] activation type (bf16 for MOE_MXFP8)
 *   w_router : device [d, E], same type
 *   dx_in    : device [T, d], same type, or NULL; dx may be dx_in (in place)
 *   dx       : device [T, d] out;  dw_router : device float32 [d, E] out
 *   ws       : device, moe_router_backward_workspace_bytes (host-only query;
 *              may be 0: then ws may be NULL)
 * Tensors are 16-byte aligned.  Sums run in a fixed order.  Errors:
 * MOE_ERR_NULL, MOE_ERR_WORKSPACE, MOE_ERR_ARG for an unaligned pointer or
 * dx == x. */
int32_t moe_router_backward_workspace_bytes(const moe_problem* p, size_t* bytes);
int32_t moe_router_backward(const moe_problem* p, const float* dlogits, const void* x, const void* w_router,
                            const void* dx_in, void* dx, float* dw_router, void* ws, size_t ws_bytes, void* stream);

/* moe_backward with another gradient for the logits: dlogits_aux [T, E]
 * float32 (moe_balance_loss_backward's), or NULL, is added to dlogits, and for
 * the learned router dx and dw_router are the gradients of the router's
 * product from that sum (dense, as moe_router_backward).  xq: the codes given
 * to moe_forward_quantized when that was the forward, else NULL.  Other
 * arguments as moe_backward; ws_bytes >= moe_backward_aux_workspace_bytes.
 * With both NULL it is moe_backward.  Errors: as moe_backward; MOE_ERR_DTYPE /
 * MOE_ERR_SHAPE for xq on a problem moe_forward_quantized does not take;
 * MOE_ERR_ARG for an unaligned xq (16), for dlogits_aux == dlogits, with
 * dlogits_aux for dlogits, w_router, x, dx or ws not 16-byte aligned, and with
 * dlogits_aux or xq for dx == x where the router is learned. */
int32_t moe_backward_aux_workspace_bytes(const moe_problem* p, size_t* bytes);
int32_t moe_backward_aux(const moe_problem* p, const void* dy, const void* x, const void* w_router,
                         const void* packed_w, const void* packed_bwd, const int32_t* topk_idx,
                         const float* topk_gate, const int32_t* offsets, const int32_t* pos, const void* fwd_ws,
                         size_t fwd_ws_bytes, void* dx, float* dlogits, float* dw_gate, float* dw_up, float* dw_down,
                         float* dw_router, void* ws, size_t ws_bytes, void* stream, const float* dlogits_aux,
                         const uint8_t* xq);

/* ---------------------------------------------------------------- the optimizer's step
 *
 * The norm of the gradients of many tensors, and an AdamW step over them, each
 * in one launch for all tensors of the same types: the end of a training step
 * whose gradients moe_backward and the norms' backward leave in float32.  With
 * t the number of the step and factor the clipping factor (1 without):
 *   g' = factor g,  m = beta1 m + (1 - beta1) g',  v = beta2 v + (1 - beta2) g'^2,
 *   w = w - lr lr_scale (m / (1 - beta1^t) / (sqrt(v / (1 - beta2^t)) + eps) + weight_decay w)
 * in float32, per element.
 *
 * moe_param, one tensor of n elements (contiguous, any shape; n = 0 is passed
 * over).  Device pointers, 16-byte aligned (scales 4):
 *   weight  : [n] w_dtype (MOE_F32 or MOE_BF16), in and out; NULL with master,
 *             m, v and the scales: a gradient for moe_grad_norm only
 *   grad    : [n] g_dtype (MOE_F32 or MOE_BF16)
 *   master  : [n] float32, in and out, or NULL.  For MOE_BF16 weights: the step
 *             is made on it and weight is its nearest bfloat16.  A MOE_BF16
 *             weight without it is rounded stochastically (below)
 *   m, v    : [n] moments, in and out, zero before the first step.  Without
 *             scales float32.  With m_scale and v_scale ([ceil(n / 128)] float32)
 *             8 bits an element: E4M3 codes whose values, times the scale of
 *             their 128 consecutive elements, are m and sqrt(v)
 *
 * 8-bit moments: a block's scale is amax / 448 (amax over its finite values; 0
 * for a block below 2^-100); a value x has the E4M3 code floor(c + f + (r + 1/2) / 2^16)
 * with its sign, at most 126, for c the code at or below 448 |x| / amax, f the
 * part of the way to the next code's value.  The quotients are float32 products
 * with float32 reciprocals, amax (1 / 448) and |x| (448 (1 / amax)), each rounded,
 * so that a scale may be a step beside the nearest.  r is the low (m) or high (v)
 * 16 bits of
 *   mix(K + i 0x9E3779B9),  K = mix(mix(mix(mix(t) ^ seed) + tensor) ^ block),
 * i the element's place in its block, tensor the place in the list, mix the
 * 32-bit finalizer of MurmurHash3.  The code of a positive sqrt(v) is at least 1,
 * that is amax / 229376: smaller roots are held that large, and their elements'
 * steps are smaller for it.  Infinite and NaN values have the NaN code.
 * A MOE_BF16 weight without master: its float32 bits plus the low 16 bits of
 * mix(that number + 0x7F4A7C15), cut to bfloat16.
 *
 * moe_param_table: writes the table that the calls read, moe_param_table_bytes()
 * bytes, to host memory and describes it in *plan (host only, no GPU call).  The
 * caller copies it to device memory, 16-byte aligned, before the first call and
 * keeps it, and the tensors where they are, as long as calls use it.  The calls
 * keep counters and partial sums in it: calls that share a table must not
 * overlap.  Errors: MOE_ERR_NULL (params, a grad, weight without m or v or the
 * reverse, one scale without the other), MOE_ERR_DTYPE (types; a master for
 * MOE_F32 weights), MOE_ERR_SHAPE (count < 1, n < 0, n >= 2^38, 2^42 elements in
 * all), MOE_ERR_ARG (not aligned, an infinite or NaN lr_scale or weight_decay,
 * tensors that a step writes overlapping any other), MOE_ERR_WORKSPACE
 * (table_bytes; host memory).
 *
 * moe_grad_norm: norm_clip[0] = sqrt(sum of squares of all gradients), in
 * float64, norm_clip[1] = max_norm / norm where the norm is larger than max_norm
 * (> 0, may be infinite), else 1; NaN if the norm is infinite or NaN.  Sums run
 * in a fixed order (bitwise reproducible).
 *   norm_clip : device float32 [2] out
 *
 * moe_adamw: one step of every tensor.
 *   hyper : host; betas in [0, 1), eps >= 0 (0: an element whose gradients were
 *           all 0 becomes NaN), seed of the random bits
 *   lr    : device float32 [1]
 *   clip  : device float32 [2] as moe_grad_norm writes it, or NULL.  If the
 *           factor is infinite or NaN the step is left out: nothing changes
 *   step  : device int32 [2], in and out: the number of steps taken, zero before
 *           the first, which the call counts up; the second word is not touched
 * A replayed graph takes the next step each time.  Errors: MOE_ERR_NULL,
 * MOE_ERR_ARG (betas, eps, max_norm, alignment), MOE_ERR_STATE (a plan that
 * moe_param_table did not write, for moe_adamw also one with gradients alone). */
typedef struct moe_param {
    void* weight;
    const void* grad;
    float* master;
    void* m;
    void* v;
    float* m_scale;
    float* v_scale;
    int64_t n;
    int32_t w_dtype;
    int32_t g_dtype;
    float lr_scale;
    float weight_decay;
} moe_param;

typedef struct moe_param_plan {
    int32_t first[14];      /* chunks of each kind of tensor begin here */
    uint32_t check;
    uint64_t descs, map;    /* offsets in the table */
    uint64_t table_bytes;
} moe_param_plan;

typedef struct moe_adamw_hyper {
    double beta1, beta2;
    float eps;
    uint32_t seed;
} moe_adamw_hyper;

int32_t moe_param_table_bytes(const moe_param* params, int32_t count, size_t* bytes);
int32_t moe_param_table(const moe_param* params, int32_t count, void* host_table, size_t table_bytes,
                        moe_param_plan* plan);
int32_t moe_grad_norm(const moe_param_plan* plan, void* table, float max_norm, float* norm_clip, void* stream);
int32_t moe_adamw(const moe_param_plan* plan, void* table, const moe_adamw_hyper* hyper, const float* lr,
                  const float* clip, int32_t* step, void* stream);

/* ---------------------------------------------------------------- a few tokens, packed weights
 *
 * moe_forward for up to MOE_FEW_MAX_TOKENS tokens on the same packed weights
 * (moe_pack_weights'), read once for all rows of an expert: what a model under
 * training is sampled and evaluated with.  Every act_dtype; MOE_MXFP8 blocks
 * take x as it is (bfloat16, not quantised) and h is not quantised either; h of
 * MOE_BF16 and MOE_MXFP8 blocks is held as two bfloat16 terms (2^-16 of it left
 * out).  No MOE_IDENTITY_EXPERTS; MOE_KEEP_GATE_UP has no effect.
 *   logits : device float32 [T, E]; input with MOE_LOGITS_GIVEN, else output
 *   mask   : device uint8 [T] or NULL; 0: the token is padding, its row of x may
 *            hold anything, its topk_idx are -1, its gates and its row of y 0
 *   topk_idx [T, k], topk_gate [T, k] : out, or NULL (kept in the workspace)
 *   y      : device [T, d] out (activation type, bfloat16 for MOE_MXFP8); may be x
 *   ws     : moe_forward_few_workspace_bytes (host-only query)
 * Ties and gates as moe_route for the same logits; a learned router's are summed in
 * another order than moe_forward's, so that two that differ by their float32
 * rounding alone may change places.  A token's result does not depend on the other
 * tokens of the call.  x, w_router, logits, packed_w, y and ws are 16-byte aligned.
 * Errors: MOE_ERR_NULL, MOE_ERR_SHAPE (T over the limit, T k max(d, H) float32 not
 * below 2^32 bytes), MOE_ERR_DTYPE, MOE_ERR_WORKSPACE, MOE_ERR_ARG for an
 * unaligned pointer. */
#define MOE_FEW_MAX_TOKENS 32
int32_t moe_forward_few_workspace_bytes(const moe_problem* p, size_t* bytes);
int32_t moe_forward_few(const moe_problem* p, const void* x, const void* w_router, float* logits, const void* packed_w,
                        const uint8_t* mask, void* y, int32_t* topk_idx, float* topk_gate, void* ws, size_t ws_bytes,
                        void* stream);

/* ---------------------------------------------------------------- a few tokens (serving)
 *
 * The block for up to MOE_DECODE_MAX_TOKENS tokens with 4-bit expert weights:
 * x and y bfloat16, h two bfloat16 terms (2^-16 of it left out), weights MXFP4
 * (OCP Microscaling v1.0: E2M1 codes, one E8M0 scale per 32 consecutive elements
 * along the contraction axis, 255 for NaN; packed with the shared exponent
 * floor(log2(amax)) - 2 clamped to [-127, 127], elements rounded to nearest even
 * and saturated to +-6, a block with a NaN given the scale 255).  act_dtype
 * MOE_BF16 or MOE_MXFP8 (no difference here), d_model and d_hidden multiples of
 * 128, no MOE_IDENTITY_EXPERTS.
 *
 * moe_pack_weights_decode quantises w_gate, w_up [E, d, H], w_down [E, H, d]
 * (device bfloat16) into packed, moe_decode_weight_bytes() bytes:
 *   W1 codes [E][2H][d/2], row n of an expert as moe_pack_weights orders them;
 *   W2 codes [E][d][H/2]; scales S1 [E][2H][d/32]; scales S2 [E][d][H/32];
 * one after the other (every region is a multiple of 256 bytes), row-major,
 * byte j of a code row holding element 2j in its low and 2j + 1 in its high
 * four bits.  Weights already in that format can be given as they are.
 *
 * moe_decode_experts: y[t] = sum_j topk_gate[t][j] FFN_e(x[t]), e =
 * topk_idx[t][j], summed in slot order in float32 and rounded once.  An index
 * outside [0, E) is a slot not in use (a padded token's row of y is zero).
 * moe_decode: router logits, top-k and gates as moe_route (bit for bit), then
 * the experts; topk_idx and topk_gate may be NULL (kept in the workspace).
 *   x [T, d] bf16; w_router [d, E] bf16 (NULL with MOE_LOGITS_GIVEN);
 *   logits float32 [T, E]; topk_idx int32 [T, k]; topk_gate float32 [T, k];
 *   y [T, d] bf16 out (not x); ws: moe_decode_workspace_bytes (host-only query)
 * x, w_router, logits, packed, y and ws are 16-byte aligned.  A token's result
 * does not depend on the other tokens of the call.  Errors: MOE_ERR_NULL,
 * MOE_ERR_SHAPE (T over the limit, d or H not a multiple of 128, T k max(d, 2 H)
 * bfloat16 not below 2^32 bytes), MOE_ERR_DTYPE, MOE_ERR_WORKSPACE, MOE_ERR_ARG
 * for an unaligned pointer or y == x. */
#define MOE_DECODE_MAX_TOKENS 256
int32_t moe_decode_weight_bytes(const moe_problem* p, size_t* bytes);
int32_t moe_decode_workspace_bytes(const moe_problem* p, size_t* bytes);
int32_t moe_pack_weights_decode(const moe_problem* p, const void* w_gate, const void* w_up, const void* w_down,
                                void* packed, void* stream);
int32_t moe_decode_experts(const moe_problem* p, const void* x, const int32_t* topk_idx, const float* topk_gate,
                           const void* packed, void* y, void* ws, size_t ws_bytes, void* stream);
int32_t moe_decode(const moe_problem* p, const void* x, const void* w_router, float* logits, const void* packed,
                   void* y, int32_t* topk_idx, float* topk_gate, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_MI355X_H */

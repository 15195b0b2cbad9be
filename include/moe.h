/*
 * moe.h -- C ABI of a single-GPU Mixture-of-Experts layer for GB300 (sm_103a),
 * forward and backward.
 *
 * The layer is the one described in "Scalable Training of Mixture-of-Experts
 * Models with Megatron Core", §2 (Megatron-Core MoE Architecture): Route
 * (router logits -> probabilities -> top-k experts, routing weights and a
 * token-expert assignment), Dispatch (permute tokens by destination expert),
 * Expert Computation (all experts' FFNs as grouped GEMMs) and Combine
 * (restore token order, weight by the gates, add a shared expert's output).
 * §5 (Selective precision) keeps the router in FP32; §5 (Kernel and shape
 * optimization) pads expert segments with zero rows to aligned sizes; §7
 * (Load Balancing) lists dropless dispatch, which is the only mode here.
 *
 * Formulas (the pages print none; these are the plain readings):
 *   z = x Wr + b                     (fp32; b optional, per expert)
 *   softmax: p = softmax(z);  sigmoid: s = 1 / (1 + exp(-z))
 *   S_t = the k experts with the largest score, slots in descending score
 *   g_tj = score_{e_tj} / sum_{i in S_t} score_i
 *   expert e (SwiGLU): a = x Wg_e, u = x Wu_e, h = silu(a) u, y_e = h Wd_e
 *   y_t = sum_j g_tj y_{e_tj}(x_t) + shared(x_t)
 * The backward returns the gradient of sum(dY * y) with the routing held
 * fixed; no gradient flows to b.
 *
 * Conventions for every entry point:
 *   - All tensor pointers are DEVICE pointers on the plan's device, row-major,
 *     16-byte aligned, owned by the caller. The library never allocates,
 *     frees or keeps device memory; the plan holds host state only.
 *   - Work is enqueued on `stream` (a cudaStream_t) and returns without
 *     synchronising. No call copies device data to the host, so forward and
 *     backward can be captured in a CUDA graph.
 *   - Arguments are validated before anything is enqueued; on any error
 *     nothing is launched and the status says why.
 *   - Errors detected on the device (a pipeline wait that timed out) are
 *     written to a status word at the start of the workspace; read them
 *     with moe_read_status.
 *   - Calls on different streams must use different workspaces.
 */
#ifndef MOE_GB300_H
#define MOE_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_ABI_VERSION 3

typedef enum {
    MOE_OK = 0,
    MOE_ERR_INVALID_ARG = 1,          /* null pointer, bad size or enum     */
    MOE_ERR_UNSUPPORTED = 2,          /* valid request the library cannot run */
    MOE_ERR_MISALIGNED = 3,           /* a pointer is not 16-byte aligned    */
    MOE_ERR_WORKSPACE_TOO_SMALL = 4,  /* saved or workspace buffer too small */
    MOE_ERR_CUDA = 5,                 /* a CUDA runtime call failed          */
    MOE_ERR_DEVICE_TIMEOUT = 6        /* a device-side wait ran out          */
} moe_status_t;

typedef enum { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 } moe_score_t;

/* Storage and arithmetic type of activations and expert weights.
 *   MOE_FP32: fp32 storage, fp32 FMA arithmetic throughout.
 *   MOE_BF16: bf16 storage, tensor-core GEMMs with fp32 accumulation.
 *   MOE_FP8_BLOCK: bf16 activations, weights and gradients; every expert
 *     GEMM runs on E4M3 operands with fp32 block scales (1x128 blocks along
 *     K for the operand indexing output rows, 128x128 for the other), fp32
 *     accumulation ("Scalable Training of Mixture-of-Experts Models with
 *     Megatron Core", §5, blockwise FP8). The router stays fp32. Layers with
 *     a shared expert are not supported in this mode (MOE_ERR_UNSUPPORTED).
 *   MOE_MXFP8: bf16 activations, weights and gradients; every expert GEMM
 *     runs on E4M3 operands in the MXFP8 recipe ("Scalable Training of
 *     Mixture-of-Experts Models with Megatron Core", §5 Platform-specific
 *     recipes: the default FP8 recipe on Blackwell, 1x32 granularity): each
 *     32 consecutive values along the GEMM's contraction dimension share one
 *     power-of-two scale 2^e (an UE8M0 byte), e the smallest integer with
 *     amax <= 448 2^e; the tensor cores apply the scales. Both operands of
 *     every GEMM are blocked along K, so weights (and the activations and
 *     gradients that feed two GEMMs) are quantised once per orientation.
 *     The router stays fp32. A shared expert runs through the same engine
 *     as a dense group of the T rows; its weights are quantised by every
 *     forward (the weight cache holds the routed experts' weights).
 *   MOE_NVFP4: as MOE_MXFP8, with every expert GEMM on NVFP4 operands
 *     ("Scalable Training of Mixture-of-Experts Models with Megatron Core",
 *     §5 Platform-specific recipes: NVFP4 for Blackwell): E2M1 values, one
 *     unsigned E4M3 scale per 16 values along K and one fp32 scale
 *     S = 2688 / amax per tensor -- one expert's part of a grouped operand
 *     (or a dense operand), with the gate and up projections [W_gate | W_up]
 *     and their output gradients one tensor each; the tensor cores apply the
 *     block scales (tcgen05.mma.kind::mxf4nvf4, .scale_vec::4X) and the GEMM
 *     epilogue divides out the two tensor scales. Requires H, F and Fs to be
 *     multiples of 256. */
typedef enum { MOE_FP32 = 0, MOE_BF16 = 1, MOE_FP8_BLOCK = 2, MOE_MXFP8 = 3, MOE_NVFP4 = 4 } moe_dtype_t;

typedef struct {
    int H;       /* hidden size; multiple of 128                          */
    int E;       /* routed experts, 1..256                                  */
    int F;       /* routed expert FFN width; multiple of 128                */
    int Fs;      /* shared expert FFN width; 0 = no shared expert, else a
                    multiple of 128                                         */
    int top_k;   /* experts per token, 1..min(E, 8)                         */
    int T_max;   /* largest token count a call may pass, >= 1               */
    int score;   /* moe_score_t                                             */
    int dtype;   /* moe_dtype_t                                             */
    unsigned flags; /* 0, or MOE_FLAG_STAGE_TIMING | MOE_FLAG_FOLD_GATES    */
    float capacity_factor; /* 0 = dropless. > 0: capacity-limited dropping
                    ("Scalable Training of Mixture-of-Experts Models with
                    Megatron Core", §7 Load Balancing): expert e computes at
                    most C = ceil(capacity_factor * T * top_k / E) of the
                    (token, slot) assignments it received, the earliest tokens
                    first; a dropped assignment adds nothing to y, gets no
                    expert gradient and has dg = 0 (its routing gradient still
                    flows through the other slots' renormalised gates).
                    In the FP8 recipes a dropped assignment never reaches its
                    expert: its rows are zeros in every quantisation block
                    along the tokens (the weight-gradient operands). */
} moe_config_t;

/* Plan flag: bracket every kernel launch of moe_forward / moe_backward with
 * CUDA events on the call's stream, for moe_stage_times. A plan with this
 * flag must not be used by two host threads at once. */
#define MOE_FLAG_STAGE_TIMING 1u

/* Plan flag: memory-efficient permutation ("Scalable Training of
 * Mixture-of-Experts Models with Megatron Core", §4, Memory-Efficient
 * Permutation: an algebraic rearrangement that drops intermediate tensors).
 * The routing weight g of each routed row is folded into its activation
 * before fc2 (h' = g silu(a) u), so fc2 yields g y_e directly and Combine is
 * a plain sum; the backward pass forms dg = <dh', h> in the fc2-dgrad
 * epilogue and recomputes h' = g h from the saved a, u for the fc2 weight
 * gradient. Results equal the unfolded layer up to rounding; the saved
 * buffer no longer holds h or the permuted expert outputs (R_pad x (F + H)
 * elements less, R_pad = routed rows padded to 128 per expert), which move
 * to the workspace. */
#define MOE_FLAG_FOLD_GATES 2u

/* Per-stage device time accumulated since the previous moe_stage_times. */
typedef struct {
    char  name[24];   /* stage, e.g. "fc1_swiglu", "fc1_wgrad", "combine"  */
    int   launches;   /* kernel launches of this stage                      */
    float total_ms;   /* summed event-timed duration of those launches      */
} moe_stage_time_t;

typedef struct moe_plan_s* moe_plan_t;

/* Opaque CUDA stream handle; pass a cudaStream_t (0 = legacy default). */
typedef struct CUstream_st* moe_stream_t;

/* Forward arguments. Element type "act" = fp32 for MOE_FP32, bf16 for
 * MOE_BF16. Optional outputs may be NULL. */
typedef struct {
    const void*  x;        /* T×H act: token hidden states                */
    const float* Wr;       /* H×E fp32: router weight                      */
    const float* b;        /* E fp32 router logit bias, or NULL            */
    const void*  W_gate;   /* E×H×F act                                    */
    const void*  W_up;     /* E×H×F act                                    */
    const void*  W_down;   /* E×F×H act                                    */
    const void*  Ws_gate;  /* H×Fs act (NULL iff Fs == 0)                   */
    const void*  Ws_up;    /* H×Fs act                                      */
    const void*  Ws_down;  /* Fs×H act                                      */
    void*        y;        /* out, T×H act                                  */
    int32_t*     topk_idx; /* optional out, T×k: chosen experts, slot order */
    float*       gates;    /* optional out, T×k: renormalised gates         */
    int32_t*     counts;   /* optional out, E: tokens per expert            */
    int32_t*     offsets;  /* optional out, E+1: first padded row of each
                              expert's segment (segments padded to 128 rows) */
    int32_t*     row_of;   /* optional out, T×k: padded row of (t, j)        */
    const int32_t* replay_topk; /* optional in, T×k: router replay (§10, RL
                              post-training) — expert of each (t, j) taken
                              from here instead of the top-k selection; the
                              logits, scores and gates are computed as usual
                              over the given experts (gates = their scores
                              over the sum of their scores). Indices outside
                              [0, E) are clamped and reported as
                              MOE_ERR_INVALID_ARG in the status word. */
    const void*  weight_cache; /* optional in (quantised-expert plans:
                              FP8_BLOCK, MXFP8, NVFP4): expert weights
                              quantised by moe_quantize_weights. When given,
                              W_gate, W_up and W_down are not read (they may
                              be NULL) and the call quantises none of the
                              routed experts' weights (an MXFP8 or NVFP4
                              layer's shared expert weights are still read and
                              quantised);
                              the matching moe_backward must be given the same
                              cache. Other dtypes: must be NULL. */
} moe_fwd_args_t;

/* Backward arguments. Gradients are overwritten (not accumulated); experts
 * that received no token get zero weight gradients. */
typedef struct {
    const void*  dY;       /* T×H act: gradient of the layer output         */
    const void*  x;        /* the forward's x                                */
    const float* Wr;       /* the forward's router weight                     */
    const void*  W_gate;   /* the forward's expert weights                    */
    const void*  W_up;
    const void*  W_down;
    const void*  Ws_gate;  /* the forward's shared-expert weights (or NULL)   */
    const void*  Ws_up;
    const void*  Ws_down;
    void*        dX;       /* out, T×H act                                   */
    float*       dWr;      /* out, H×E fp32                                  */
    void*        dW_gate;  /* out, E×H×F act                                 */
    void*        dW_up;    /* out, E×H×F act                                 */
    void*        dW_down;  /* out, E×F×H act                                 */
    void*        dWs_gate; /* out, H×Fs act (NULL iff Fs == 0)                */
    void*        dWs_up;
    void*        dWs_down;
    const void*  weight_cache; /* quantised recipes: the cache given to the
                              forward (W_gate, W_up, W_down then unread), or
                              NULL when the forward quantised the bf16
                              weights itself. Other dtypes: NULL. */
} moe_bwd_args_t;

/* Validate `cfg` for `device` and build a plan (host memory only).
 * Errors: INVALID_ARG (null, sizes out of range, unknown flags,
 *         capacity_factor negative or not finite),
 *         UNSUPPORTED (dtype not built, device not sm_103, MOE_FP8_BLOCK
 *         with a shared expert, MOE_NVFP4 with H, F or Fs not a multiple of
 *         256), CUDA. */
moe_status_t moe_plan_create(const moe_config_t* cfg, int device, moe_plan_t* out);

/* Free a plan. NULL is accepted. */
moe_status_t moe_plan_destroy(moe_plan_t plan);

/* Bytes of the two caller-owned buffers for a call with T tokens:
 *   saved: written by moe_forward, read by moe_backward (routing, permuted
 *          activations and FFN intermediates of that forward);
 *   ws:    scratch for either call; its first 256 bytes hold the status word.
 * Errors: INVALID_ARG (null, T < 1 or T > T_max). */
moe_status_t moe_workspace_size(moe_plan_t plan, int T, size_t* saved_bytes, size_t* ws_bytes);

/* Enqueue the forward pass for T tokens: Route, Dispatch, Expert
 * Computation, Combine. Writes args->y, the optional outputs and `saved`.
 * Errors: INVALID_ARG, MISALIGNED, WORKSPACE_TOO_SMALL, CUDA. */
moe_status_t moe_forward(moe_plan_t plan, int T, const moe_fwd_args_t* args,
                         void* saved, size_t saved_bytes, void* ws, size_t ws_bytes,
                         moe_stream_t stream);

/* Enqueue the backward pass for T tokens, using the `saved` buffer of the
 * forward with the same T, inputs and weights (it is only read).
 * Errors: INVALID_ARG, MISALIGNED, WORKSPACE_TOO_SMALL, CUDA. */
moe_status_t moe_backward(moe_plan_t plan, int T, const moe_bwd_args_t* args,
                          const void* saved, size_t saved_bytes, void* ws, size_t ws_bytes,
                          moe_stream_t stream);

/* Synchronise `stream`, then return the device status word kept in `ws`
 * (MOE_OK or MOE_ERR_DEVICE_TIMEOUT); CUDA errors give MOE_ERR_CUDA. */
moe_status_t moe_read_status(moe_plan_t plan, const void* ws, moe_stream_t stream);

/* Static, NUL-terminated description of a status code. */
const char* moe_status_string(moe_status_t status);

/* Device time per stage of every moe_forward / moe_backward enqueued since
 * the previous call (plans created with MOE_FLAG_STAGE_TIMING only; the
 * measurement covers eagerly launched calls, not graph replays). Waits for
 * the recorded events, writes up to `capacity` entries in first-launch
 * order, sets *count to the number of stages and clears the record.
 * Errors: INVALID_ARG (null, or a plan without the flag), CUDA. */
moe_status_t moe_stage_times(moe_plan_t plan, moe_stage_time_t* out, int capacity, int* count);

/* Routing without a caller-provided workspace. The paper has no
 * counterpart: this entry exists for callers that cannot allocate device
 * memory -- their memory is owned by a framework pool or a budget fixed at
 * start-up, or they run in loops that must not call cudaMalloc (it can
 * synchronise the device) -- and so cannot pass the `ws` buffer that
 * moe_forward needs.
 * Computes, for T tokens, the same routing outputs as moe_forward's optional
 * outputs: topk_idx (T×k), gates (T×k), counts (E), offsets (E+1, padded
 * segment starts) and row_of (T×k), from x (T×H act), Wr (H×E fp32) and the
 * optional bias b (E fp32). A capacity_factor of the plan changes none of
 * them. All pointers are caller-owned device pointers, 16-byte aligned;
 * nothing is allocated or freed.
 * Scratch: a 64 MiB array inside the library's device image, held on every GPU
 * that loads the library until the process exits. A call needs about
 * 8·T·k + 8·ceil(T/32)·E + 508·min(E, T·k) bytes of it, plus up to 32·T·E
 * for E > 32 (the router's partial logits over at most 8 splits of H); larger
 * T returns MOE_ERR_WORKSPACE_TOO_SMALL before anything is launched.
 * The first call on a device looks up the array's device address (once per
 * device, with that device current); make that first call before any
 * stream capture. The address is kept for the life of the process: after a
 * cudaDeviceReset (or any other teardown of the device's primary context)
 * it is stale, and neither this entry point nor a plan created before the
 * reset may be used again on that device. All calls share the array and it keeps the last call's
 * contents (every entry a call reads is written earlier in the same call);
 * calls whose work overlaps on the GPU -- from different streams or host
 * threads -- race on it and must be serialised by the caller.
 * Errors: INVALID_ARG, MISALIGNED, WORKSPACE_TOO_SMALL, CUDA. */
moe_status_t moe_route_static(moe_plan_t plan, int T, const void* x, const float* Wr,
                              const float* b, int32_t* topk_idx, float* gates, int32_t* counts,
                              int32_t* offsets, int32_t* row_of, moe_stream_t stream);

/* Blockwise E4M3 quantiser used by the MOE_FP8_BLOCK layer, on a row-major
 * rows x cols bf16 device matrix (both multiples of 128). Scale of a block =
 * amax / 448 in fp32 (1 for an all-zero block); codes are E4M3 of
 * value / scale, rounded to nearest even and saturated ("Scalable Training of
 * Mixture-of-Experts Models with Megatron Core", §5, blockwise FP8).
 *   MOE_Q_ROWS:    1x128 blocks along rows: codes rows x cols,
 *                  scales rows x cols/128.
 *   MOE_Q_TILES:   128x128 blocks: codes rows x cols, scales (rows/128) x
 *                  (cols/128).
 *   With MOE_Q_ROWS or MOE_Q_TILES, when codes_t and scales_t are both
 *   given, the same pass also writes the 128x128-block codes of the
 *   transpose, codes_t cols x rows with scales_t (cols/128) x (rows/128)
 *   (the layer quantises its gradients this way, reading them once).
 *   MOE_Q_COLS_T:  per column over 128-row blocks, transposed output:
 *                  codes_t cols x rows, scales_t cols x rows/128.
 *   MOE_Q_TILES_T: 128x128 blocks, transposed output: codes_t cols x rows,
 *                  scales_t (cols/128) x (rows/128).
 * Unused outputs may be NULL. Enqueued on `stream`.
 * Errors: INVALID_ARG, MISALIGNED, CUDA. */
enum { MOE_Q_ROWS = 0, MOE_Q_TILES = 1, MOE_Q_COLS_T = 2, MOE_Q_TILES_T = 3 };
moe_status_t moe_fp8_quantize(int rows, int cols, int mode, const void* in, uint8_t* codes,
                              float* scales, uint8_t* codes_t, float* scales_t, moe_stream_t stream);

/* Quantised expert weights for MOE_FP8_BLOCK, MOE_MXFP8 and MOE_NVFP4 plans ("Scalable Training of
 * Mixture-of-Experts Models with Megatron Core", §5 Kernel and shape
 * optimization: grouped quantization of the experts' weights, done once
 * and kept). A caller that keeps E4M3 weights between steps -- they change
 * once per optimizer step, while a step may run several forward/backward
 * passes -- quantises them once into a caller-owned device buffer, the
 * weight cache, and passes it as weight_cache to moe_forward and
 * moe_backward, which then skip their own weight quantisation.
 *
 * moe_weight_cache_size: bytes of the cache for this plan (0 for plans
 * without quantised experts). Errors: INVALID_ARG.
 *
 * moe_quantize_weights: quantise W_gate, W_up (E x H x F bf16) and W_down
 * (E x F x H bf16) into `cache` (cache_bytes >= the size above), enqueued
 * on `stream`. The cache holds each matrix's E4M3 codes in its own layout
 * with the plan's scales (MOE_FP8_BLOCK: one fp32 scale per 128x128 block,
 * amax / 448, 1 for an all-zero block; MOE_MXFP8: the codes of both
 * orientations, each with its UE8M0 scale per 32 values; MOE_NVFP4: the
 * E2M1 codes of both orientations with their E4M3 scales per 16 values, and
 * each expert's tensor maxima of [W_gate | W_up] and W_down), exactly the codes
 * the layer would produce inside moe_forward; its internal layout is
 * private to the library version. 16-byte aligned device pointers, owned by
 * the caller.
 * Errors: INVALID_ARG (null), UNSUPPORTED (plan has no quantised experts),
 * MISALIGNED, WORKSPACE_TOO_SMALL (cache_bytes), CUDA. */
moe_status_t moe_weight_cache_size(moe_plan_t plan, size_t* bytes);
moe_status_t moe_quantize_weights(moe_plan_t plan, const void* W_gate, const void* W_up,
                                  const void* W_down, void* cache, size_t cache_bytes,
                                  moe_stream_t stream);

/* MXFP8 quantiser used by the MOE_MXFP8 layer, on a row-major rows x cols
 * bf16 device matrix (both multiples of 128). Blocks of 32 values share the
 * scale 2^e, e the smallest integer with amax <= 448 2^e, clamped to
 * [-127, 127] (-127 for an all-zero block), stored as the UE8M0 byte
 * e + 127; a value is stored as the E4M3 code of v 2^-e (round to nearest
 * even). Scales are written as "scale atoms", the layout the GEMMs copy into
 * tensor memory: for an operand read as [n][K], one 512-byte atom per
 * 128-row tile t and 128-deep K block b at (t * K/128 + b) * 512, whose byte
 * 16 (m % 32) + 4 (m / 32) + j holds the scale of tile row m and 32-deep
 * sub-block j.
 *   codes, scales (optional): blocks along the rows; codes rows x cols,
 *     atoms of the [rows][K = cols] operand (rows * cols / 32 bytes).
 *   codes_c, scales_c (optional): blocks down the columns (32 rows each);
 *     col_transposed 1: codes cols x rows (the transpose), col_transposed 0:
 *     codes rows x cols in place; atoms of the [cols][K = rows] operand.
 * At least one pair must be given. Enqueued on `stream`.
 * Errors: INVALID_ARG, MISALIGNED, CUDA. */
moe_status_t moe_mx_quantize(int rows, int cols, const void* in, uint8_t* codes, uint8_t* scales,
                             uint8_t* codes_c, uint8_t* scales_c, int col_transposed, moe_stream_t stream);

/* NVFP4 quantiser used by the MOE_NVFP4 layer, on a row-major rows x cols
 * bf16 device matrix (both multiples of 128) taken as one tensor: its
 * largest magnitude goes to *amax (a device float, overwritten), the tensor
 * scale is S = 2688 / amax (1 for an all-zero matrix), and each block of
 * 16 values gets the E4M3 scale sb = E4M3(a S / 6) (a the block's largest
 * magnitude; s its value) and the E2M1 codes of v (S / s) (nearest, ties to
 * the even code, saturating at 6; zero codes when s = 0), every step an
 * fp32 operation rounded to nearest even. Codes are packed two per byte,
 * the lower-index value in the low 4 bits. Scale atoms: for an operand read
 * as [n][K], one 512-byte atom per 128-row tile t and 64-value K chunk b at
 * (t * K/64 + b) * 512, whose byte 16 (m % 32) + 4 (m / 32) + j holds the
 * scale of tile row m and 16-value sub-block j.
 *   codes, scales (optional): blocks along the rows; codes rows x cols/2
 *     bytes, atoms of the [rows][K = cols] operand (rows * cols / 16 bytes).
 *   codes_t, scales_t (optional): blocks down the columns (16 rows each),
 *     codes of the transpose, cols x rows/2 bytes; atoms of the
 *     [cols][K = rows] operand.
 * At least one pair must be given. Enqueued on `stream`.
 * Errors: INVALID_ARG, MISALIGNED, CUDA. */
moe_status_t moe_nv_quantize(int rows, int cols, const void* in, float* amax, uint8_t* codes, uint8_t* scales,
                             uint8_t* codes_t, uint8_t* scales_t, moe_stream_t stream);

/* Failure-detection check. Every pipelined kernel of the layer waits on
 * its shared-memory mbarriers with a bounded wait (2 s); when a wait runs out
 * the kernel records MOE_ERR_DEVICE_TIMEOUT in the status word and returns,
 * so a stalled pipeline ends with an error instead of hanging the GPU. This
 * entry point runs that wait on an mbarrier that is never signalled: after
 * the call, moe_read_status(plan, ws, stream) returns MOE_ERR_DEVICE_TIMEOUT
 * and the device stays usable. `ws` is any workspace (its status word is
 * overwritten). Errors: INVALID_ARG, CUDA. */
moe_status_t moe_diag_wait_timeout(void* ws, moe_stream_t stream);

/* Auxiliary-loss-free load balancing: one update of the per-expert router
 * logit bias ("Scalable Training of Mixture-of-Experts Models with Megatron
 * Core", §7 Load Balancing, "auxiliary-loss-free biasing"; the pages give no
 * rule): with c_e the tokens expert e received in the last forward (the
 * `counts` output) and c_mean their mean over the E experts,
 *   b_e <- b_e + rate * sign(c_mean - c_e),   sign(0) = 0,
 * so under-loaded experts become more likely to be selected and over-loaded
 * ones less. The comparison is exact (integers: E*c_e against sum of c).
 * counts: E int32, b: E fp32 (updated in place), device pointers, enqueued
 * on `stream`. Errors: INVALID_ARG (null, E outside 1..256, rate not
 * finite), CUDA. */
moe_status_t moe_update_bias(int E, const int32_t* counts, float rate, float* b, moe_stream_t stream);

/* ------------------------------------------------------------------------
 * Operators around the layer
 *
 * What a block does next to its experts: the residual addition with a
 * root-mean-square norm in front of the router, the sort of tokens by expert
 * and the way back for experts other than this library's (the routing of
 * moe_route_static, or of any router), and the global gradient norm with
 * clipping. Conventions as above, and:
 *   - they need no plan; they run on the calling thread's current device, on
 *     which the pointers and the stream must live;
 *   - "act" values are fp32 (MOE_FP32) or bf16 (MOE_BF16); any width H from
 *     1 to 2^20 is accepted; row strides (ld*) count elements and are at least H;
 *   - zero rows, tokens or tensors are accepted: nothing is read, outputs
 *     that do not depend on rows (weight gradients, counts, the norm) are
 *     written, and the pointers of empty tensors may be NULL;
 *   - sums, means and norms are fp32 or wider, in a fixed order: the same
 *     inputs give the same bits.
 * ------------------------------------------------------------------------ */

/* 8-bit output of moe_add_rms_norm.
 *   MOE_NORM_FP8_BLOCK: E4M3 codes (rows x H bytes) with one fp32 scale per
 *     1x128 block (rows x H/128): amax / 448, 1 for an all-zero block; codes
 *     of the fp32 quotient value / scale, nearest even, saturated, a zero's
 *     sign kept.
 *   MOE_NORM_MXFP8: E4M3 codes with one UE8M0 scale per 1x32 block, 2^e with
 *     e the smallest integer such that amax <= 448 2^e, in the scale atoms of
 *     moe_mx_quantize: ceil(rows/128) * H/128 atoms of 512 bytes; the scale
 *     bytes of rows past the last one in the last tile are written as 0.
 * Both quantise the fp32 norm, before any rounding to act. They need H to be
 * a multiple of 128 and row strides that are multiples of 16 bytes. */
enum { MOE_NORM_PLAIN = 0, MOE_NORM_FP8_BLOCK = 1, MOE_NORM_MXFP8 = 2 };

typedef struct {
    const void*  x;        /* rows x H act, row stride ldx                   */
    const void*  residual; /* rows x H act, row stride ldr, or NULL          */
    const float* weight;   /* H fp32                                         */
    void*        h;        /* optional out (with a residual): x + residual;
                              may be x or residual itself                    */
    void*        y;        /* out, rows x H act: the norm (optional with an
                              8-bit output); may be x or residual itself     */
    float*       rstd;     /* optional out, rows: 1 / rms, for the backward  */
    uint8_t*     codes;    /* 8-bit output (NULL for MOE_NORM_PLAIN)         */
    void*        scales;
    long long    ldx, ldr, ldh, ldy;
} moe_norm_fwd_args_t;

/* s = x + residual (fp32), rstd = (mean(s^2) + eps)^(-1/2), y = s rstd weight.
 * h is s rounded to act; the norm is that of the unrounded sum.
 * Errors: INVALID_ARG (null or missing pointers, rows < 0, H < 1, a stride
 * below H, unknown dtype or quant, eps negative or not finite, an 8-bit
 * output with H not a multiple of 128), MISALIGNED (a pointer, or a stride
 * with an 8-bit output), CUDA. */
moe_status_t moe_add_rms_norm(int rows, int H, int dtype, int quant, float eps,
                              const moe_norm_fwd_args_t* args, moe_stream_t stream);

typedef struct {
    const void*  dy;       /* rows x H act: gradient of y                     */
    const void*  h;        /* rows x H act: the normalised sum (h, or x)       */
    const float* rstd;     /* rows: the forward's                              */
    const float* weight;   /* H fp32                                           */
    const void*  dh;       /* rows x H act: gradient that reaches h from the
                              residual stream, or NULL                         */
    void*        dx;       /* out, rows x H act: gradient of x, and of the
                              residual; may be dy or dh itself                 */
    float*       dweight;  /* optional out, H fp32 (overwritten)               */
    long long    lddy, ldh, lddh, lddx;
} moe_norm_bwd_args_t;

/* With n = h rstd and c = mean(weight dy n) over the row:
 *   dx = rstd (weight dy - n c) + dh,   dweight = sum over rows of dy n.
 * ws (moe_norm_workspace_size bytes, scratch for dweight's partial sums) may
 * be NULL when dweight is NULL.
 * Errors: as the forward's, and WORKSPACE_TOO_SMALL. */
moe_status_t moe_norm_workspace_size(int rows, int H, size_t* ws_bytes);
moe_status_t moe_add_rms_norm_backward(int rows, int H, int dtype, const moe_norm_bwd_args_t* args,
                                       void* ws, size_t ws_bytes, moe_stream_t stream);

/* Tokens sorted by expert. Slot t k + j is the j-th choice of token t; its
 * expert is topk[t][j], and any value outside [0, E) drops the slot. Expert
 * e's segment starts at row offsets[e] (a multiple of `align`), holds its
 * slots in ascending order, and is padded to the next multiple of `align`.
 * moe_sort_rows_cap gives the rows that any routing of T tokens fits in,
 * T k + min(E, T k) (align - 1) rounded up to align; buffers of rows have
 * at least that many.
 * moe_sort_index writes
 *   counts (E):      kept slots of each expert,
 *   offsets (E + 1): first row of each segment; offsets[E] rows are in use,
 *   row_of (T x k):  the row of each slot, -1 if dropped,
 *   slot_of (rows):  the slot of each row, -1 for padding and unused rows.
 * Limits: 1 <= k <= 32, 1 <= E <= 1024, 1 <= align <= 4096, rows < 2^31.
 * Errors: INVALID_ARG, MISALIGNED, CUDA. */
moe_status_t moe_sort_rows_cap(int T, int k, int E, int align, long long* rows);
moe_status_t moe_sort_index(int T, int k, int E, int align, const int32_t* topk, int32_t* counts,
                            int32_t* offsets, int32_t* row_of, int32_t* slot_of, long long rows,
                            moe_stream_t stream);

/* The index that the three calls below move rows by (moe_sort_index's, or
 * moe_route_static's row_of and offsets). Rows outside [0, rows) in row_of
 * are dropped slots. The routing tables of moe_forward and moe_route_static
 * give every slot a row: a plan with a capacity_factor drops by the row's place
 * in its segment and does not mark it there. To move rows as such a plan does,
 * set row_of to -1 first wherever
 *     row_of - offsets[expert] >= ceil(capacity_factor T k / E). */
typedef struct {
    int T, k, H, dtype;      /* dtype MOE_FP32 or MOE_BF16                     */
    long long rows;          /* rows of the sorted buffer                      */
    const int32_t* row_of;   /* T x k                                          */
    const int32_t* slot_of;  /* rows, or NULL: padding rows are not written    */
    const int32_t* in_use;   /* one device int, the rows in use (offsets + E);
                                needed with slot_of, 4-byte aligned            */
} moe_sorted_t;

/* Xp[row_of[t][j]] = x[t]; the padding rows (slot_of < 0) below *in_use are
 * zeros, rows from there on are not written. The gradient of x is
 * moe_unsort_rows of the rows' gradients without gates.
 * Errors: INVALID_ARG, MISALIGNED, CUDA. */
moe_status_t moe_sort_rows(const moe_sorted_t* index, const void* x, long long ldx, void* Xp,
                           long long ldp, moe_stream_t stream);

/* y[t] = residual[t] + sum_j gates[t][j] Yp[row_of[t][j]], fp32 in slot order,
 * rounded once. gates (T x k fp32) and residual (T x H act) may be NULL
 * (weights 1, residual 0); y may be residual itself.
 * Errors: INVALID_ARG, MISALIGNED, CUDA. */
moe_status_t moe_unsort_rows(const moe_sorted_t* index, const void* Yp, long long ldp,
                             const float* gates, const void* residual, long long ldr, void* y,
                             long long ldy, moe_stream_t stream);

/* Gradient of moe_unsort_rows with respect to Yp and gates (that of the
 * residual is dY): dYp[row_of[t][j]] = gates[t][j] dY[t], the padding rows as
 * in moe_sort_rows; dgates[t][j] = <dY[t], Yp[row_of[t][j]]>, 0 for a dropped
 * slot. dgates may be NULL (Yp may then be NULL too); dYp may be Yp itself.
 * Errors: INVALID_ARG, MISALIGNED, CUDA. */
moe_status_t moe_unsort_rows_backward(const moe_sorted_t* index, const void* dY, long long lddy,
                                      const void* Yp, long long ldp, const float* gates, void* dYp,
                                      long long ldd, float* dgates, moe_stream_t stream);

/* One gradient tensor of moe_clip_grad_norm: n values at g, clipped into out
 * (NULL: not written; may be g itself). Pointers need the alignment of their
 * type only, so views into one flat buffer are fine. Tensors do not overlap. */
typedef struct {
    const void* g;
    void*       out;
    long long   n;
    int         dtype;      /* MOE_FP32 or MOE_BF16 */
    int         reserved;   /* 0 */
} moe_grad_t;

/* Global gradient norm over `count` tensors and clipping by it:
 *   norm = sqrt(sum of g^2 over every value of every tensor),
 *   out = g min(1, max_norm / norm)   (fp32 product, rounded once).
 * max_norm > 0; infinity clips nothing. A norm that is infinite (in fp32) or
 * NaN leaves the values as they are (out = g): the caller sees it in *norm and
 * skips the step. The sum carries more bits than fp32 has (and all of its range in 64
 * bits), so the norm and max_norm / norm are the nearest fp32 values. `list` is a
 * host array, read during the call; *norm is a device float.
 * Errors: INVALID_ARG (also a norm of more than 2^46 bytes), MISALIGNED,
 * WORKSPACE_TOO_SMALL, CUDA. */
moe_status_t moe_clip_workspace_size(int count, size_t* ws_bytes);
moe_status_t moe_clip_grad_norm(int count, const moe_grad_t* list, float max_norm, float* norm,
                                void* ws, size_t ws_bytes, moe_stream_t stream);

/* ------------------------------------------------------------------------
 * Products over rows sorted by expert
 *
 * What stands between moe_sort_rows and moe_unsort_rows for experts of the
 * caller's own. Conventions as above, and:
 *   - segment e holds the rows from offsets[e] on: counts[e] of them (without
 *     counts all up to offsets[e + 1]) belong to the expert, the others up to
 *     offsets[e + 1] are padding. offsets and counts are moe_sort_index's or a
 *     layer's, read on the device; what they hold is clamped to the row buffers;
 *   - padding rows of an input are not read and those of an output are written
 *     as zeros; rows past the last segment are neither read nor written;
 *   - each value depends on its own row (or expert) alone: infinities and NaN
 *     elsewhere do not reach it;
 *   - an output overlaps no input and no other output (the same pointer is
 *     INVALID_ARG);
 *   - row strides (ld*) count elements and are at least a row's values, in any
 *     alignment for moe_grouped_*: operands whose pointer and strides are
 *     multiples of 16 bytes are read by TMA, others by loads that cost more.
 * ------------------------------------------------------------------------ */
typedef struct {
    int E;                   /* experts, 1..1024                               */
    int dtype;               /* MOE_FP32 or MOE_BF16                           */
    long long rows;          /* rows of the row buffers, 0..2^31 - 1024        */
    const int32_t* offsets;  /* E + 1; NULL with E = 1: one segment, all rows  */
    const int32_t* counts;   /* E, or NULL                                     */
} moe_groups_t;

/* Y[r] = X[r] W_e for the rows r of each segment e; X rows x K, Y rows x N, of
 * type groups->dtype (products of bf16 values are exact and summed in fp32 on
 * the tensor cores; fp32 values use fp32 FMAs, in pieces of 256 terms that are
 * added up), rounded once.
 * W_e[k][n] stands at W + e sw + k ldw + n, or with w_nk at W + e sw + n ldw + k
 * (weights stored out x in). The gradient of X is the same call on dY with the
 * other w_nk and K and N exchanged.
 * Errors: INVALID_ARG (null pointers, sizes out of range, K or N outside
 * 1..2^20, a stride below a row's values, sw below an expert's), MISALIGNED (a
 * pointer not on a 16-byte boundary; offsets and counts 4), CUDA. */
moe_status_t moe_grouped_matmul(const moe_groups_t* groups, int K, int N, const void* X, long long ldx,
                                const void* W, long long ldw, long long sw, int w_nk, void* Y, long long ldy,
                                moe_stream_t stream);

/* D_e[m][n] = sum over the expert's rows r of A[r][m] B[r][n], overwritten, zeros
 * for an expert without rows; A rows x M, B rows x N, D_e[m][n] at D + e sd +
 * m ldd + n, of type groups->dtype. With A = X and B = dY it is the gradient of
 * W (K x N); with A = dY and B = X that of weights stored out x in.
 * Errors: as moe_grouped_matmul. */
moe_status_t moe_grouped_wgrad(const moe_groups_t* groups, int M, int N, const void* A, long long lda,
                               const void* B, long long ldb, void* D, long long ldd, long long sd,
                               moe_stream_t stream);

/* The product on E4M3 codes with fp32 scales of 128 values: A is rows x K codes
 * with one scale per 1x128 block (SA rows x K/128: moe_add_rms_norm's, moe_quantize_rows'
 * or moe_fp8_quantize's), B_e K x N codes with one per 128x128 tile (moe_fp8_quantize
 * with MOE_Q_TILES over the E K x N weights), K a multiple of 128, N any:
 *   Y[r][n] = sum_kb SA[r][kb] SB_e[kb][n/128] sum_{k in block kb} A[r][k] B_e[k][n],
 * code products and their sums of 128 in fp32 on the tensor cores, the scaled sums in
 * fp32 FMAs in ascending kb, rounded once to groups->dtype. SA SB is formed first, in fp32:
 * it is infinite above 2^128 and loses bits below 2^-126, whatever the sum beside it is.
 * B_e[k][n] at B + e sb + k ldb + n with SB_e[kb][nb] at SB + e ssb + kb ldsb + nb, or
 * with b_nk B + e sb + n ldb + k and SB + e ssb + nb ldsb + kb (the transpose's view of
 * the same codes: the gradient of A's rows takes the codes of dY and this view). A dense
 * weight gradient over a multiple of 128 tokens is A = X's codes along the tokens
 * (MOE_Q_COLS_T) times B = dY's tile codes.
 * Errors: as moe_grouped_matmul, and INVALID_ARG for K not a multiple of 128,
 * MISALIGNED for lda, ldb or sb not multiples of 16. */
typedef struct {
    const uint8_t* A;  long long lda;
    const float*   SA; long long ldsa;
    const uint8_t* B;  long long ldb, sb;
    const float*   SB; long long ldsb, ssb;
    int            b_nk;
    void*          Y;  long long ldy;
} moe_fp8_matmul_args_t;
moe_status_t moe_fp8_matmul(const moe_groups_t* groups, int K, int N, const moe_fp8_matmul_args_t* args,
                            moe_stream_t stream);

/* E4M3 codes of activation rows, any number of them: one fp32 scale per 1x128 block,
 * amax / 448 (1 where that is zero), codes of the fp32 quotient value / scale, nearest
 * even, saturated. x rows x K of dtype (MOE_FP32, MOE_BF16), K a multiple of 128;
 * codes rows x K (row stride ldc), scales rows x K/128 (row stride lds). With in_use
 * (one device int, e.g. offsets + E) only the rows below *in_use are read and written.
 * A NaN's code is NaN; a block that holds an infinity has an infinite scale.
 * Errors: INVALID_ARG, MISALIGNED (a pointer, or ldx or ldc not multiples of 16
 * bytes), CUDA. */
moe_status_t moe_quantize_rows(long long rows, int K, int dtype, const void* x, long long ldx, uint8_t* codes,
                               long long ldc, float* scales, long long lds, const int32_t* in_use,
                               moe_stream_t stream);

/* Synchronise `stream`, then say whether a device-side wait of the products above ran
 * out on the current device since the last such call (MOE_ERR_DEVICE_TIMEOUT: their
 * outputs since then cannot be used), as moe_read_status does for the layer. Not for
 * streams under capture. */
moe_status_t moe_products_status(moe_stream_t stream);

/* Failure-detection check of the products, as moe_diag_wait_timeout is the layer's: runs the
 * waits of their kernels on an mbarrier that is never signalled: one with a limit of 10 ms, one
 * with the usual limit that the first one's abort flag ends, and one of 4000 tries. which: the
 * row products' status word (0), the weight gradients' (1) or the 8-bit products' (2).
 * moe_products_status then returns MOE_ERR_DEVICE_TIMEOUT once, and the device stays usable.
 * Errors: INVALID_ARG, CUDA. */
moe_status_t moe_diag_products_wait(int which, moe_stream_t stream);

/* MOE_ABI_VERSION of the loaded library. */
int moe_abi_version(void);

#ifdef __cplusplus
}
#endif
#endif /* MOE_GB300_H */

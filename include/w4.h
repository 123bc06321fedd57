/*
 * w4.h -- C ABI of the int4-weight quantized linear layer for NVIDIA GB300 (sm_103a).
 *
 * The layer computes y = x . W^T with W stored as 4-bit codes q in 0..15
 * ("uint4b8": the weight value is q - 8) and a scale per group of input
 * columns, optionally plus an additive zero per group:
 *     w[k, n] = (q[k, n] - 8) * s[k / group, n]  (+ z[k / group, n])
 *
 * Sources (page title, then the section the rule comes from):
 *   [INC]  vLLM API docs, inc.schemes.inc_w4a8_linear: INCXPUW4A8LinearMethod
 *          (class docstring; create_weights; apply_weights).
 *   [CT]   vLLM v0.10.1.1 API docs, compressed_tensors_w4a8_int:
 *          CompressedTensorsW4A8Int (__init__; create_weights).
 *   [FP8]  vLLM API docs, quantization.w4afp8: W4AFP8Config (__init__;
 *          get_checkpoint_weight_mapper); _repack_signed_int4_to_uint4b8.
 *   [ZEN]  vLLM API docs, kernels.linear.mixed_precision.zentorch:
 *          ZentorchWNA16LinearKernel (can_implement; _zentorch_woq_eligible).
 *   [OMNI] vllm-omni quantization/cpu_int4.py (module docstring; pack_nibbles).
 *
 * Conventions shared by every entry point
 *   - Every tensor pointer is a DEVICE pointer owned by the caller. The library
 *     allocates no device memory and keeps no pointer after the call returns.
 *   - All matrices are row-major and contiguous. Base pointers of matrices must
 *     be 16-byte aligned; scale/zero/bias vectors 8-byte aligned.
 *   - `stream` is a cudaStream_t passed as void* (NULL = the legacy default
 *     stream). Calls are asynchronous on that stream.
 *   - Arguments are validated on the host before anything is launched. A
 *     status other than W4_OK means nothing was launched and nothing written;
 *     w4_last_error() then returns a message (per calling thread).
 *   - A call with zero rows (M == 0 or R == 0) does nothing and returns W4_OK.
 *   - N and K must be multiples of 8 ([INC] _DIM_ALIGNMENT and create_weights:
 *     both GEMM dims multiples of 8). group is -1 (one group spanning K,
 *     [CT] create_weights) or a positive divisor of K ([ZEN] can_implement).
 *     Group sizes the kernels do not tile return W4_ERR_UNSUPPORTED.
 *   - The pipelined kernels bound every wait. If a wait runs out, the kernel
 *     records W4_ERR_TIMEOUT in a device status word and returns;
 *     w4_device_status() reads and clears it.
 *   - The < 512-token choice between W4A8 and W4A16 ([INC] _MIN_TOKENS_FOR_INT8)
 *     is the caller's: the library has no dispatch between paths.
 */
#ifndef W4_H_
#define W4_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  W4_OK = 0,
  W4_ERR_NULL = 1,        /* a required pointer is NULL */
  W4_ERR_ALIGN = 2,       /* N or K not a multiple of 8, or a pointer misaligned */
  W4_ERR_GROUP = 3,       /* group is neither -1 nor a positive divisor of K */
  W4_ERR_DTYPE = 4,       /* dtype not accepted (e.g. bf16 scales to w4a8_gemm) */
  W4_ERR_UNSUPPORTED = 5, /* valid per the layer's rules but outside what the kernels tile */
  W4_ERR_SHAPE = 6,       /* negative or inconsistent sizes */
  W4_ERR_CUDA = 7,        /* a CUDA runtime call failed (message in w4_last_error) */
  W4_ERR_TIMEOUT = 8,     /* a bounded wait inside a kernel ran out */
  W4_ERR_WORKSPACE = 9    /* workspace NULL, too small or misaligned */
} w4_status;

typedef enum {
  W4_BF16 = 0,
  W4_FP16 = 1,
  W4_INT8 = 2,
  W4_FP8_E4M3 = 3
} w4_dtype;

/* Operations that take a workspace (see w4_workspace_bytes). */
typedef enum {
  W4_OP_W4A8 = 0,           /* w4a8_gemm and w4a8_group_partials */
  W4_OP_W4AFP8_MOE = 1,     /* w4afp8_moe_grouped_gemm, w4afp8_moe_gemm_bf16in (M = R, the row count) */
  W4_OP_MOE_ROUTE = 2,      /* w4_moe_route (M = T tokens, N = E experts; K = 1, group ignored) */
  W4_OP_MOE_ROUTE_GROUPED = 3, /* w4_moe_route_grouped (M = T tokens, N = E experts; K = 1, group ignored) */
  W4_OP_FP8_BLOCK = 4,      /* w4_fp8_block_gemm (group ignored) */
  W4_OP_FP8_BLOCK_IN = 5,   /* w4_fp8_block_gemm_bf16in (group = 0), w4_fp8_block_moe_gemm_bf16in (M = R rows, group = E) */
  W4_OP_FP4_IN = 6,         /* w4_fp4_gemm_bf16in (M = rows, group = 16 or 32: the format's block) */
  W4_OP_MOE_DECODE = 7,     /* w4_moe_decode (M = T tokens, N = top_k, K = I; group ignored) */
  W4_OP_FP4_MOE_IN = 8      /* w4_fp4_moe_gemm_bf16in (M = R rows, group = 16 or 32) */
} w4_op;

/* 4-bit weight formats. */
typedef enum {
  W4_FMT_MXFP4 = 0,  /* e2m1, a power of two (e8m0) per 32 columns */
  W4_FMT_NVFP4 = 1,  /* e2m1, an e4m3 scale per 16 columns, an fp32 scale per tensor */
  W4_FMT_INT4 = 2    /* uint4b8 (q - 8), an fp16 scale per group of columns */
} w4_format;

/* Router scores of w4_moe_route_grouped. */
typedef enum {
  W4_SCORE_SIGMOID = 0,
  W4_SCORE_SOFTMAX = 1
} w4_scoring;

/*
 * Bytes of device workspace an operation needs for M activation rows of
 * length K. The tensor-core GEMMs first widen the 8-bit activations once into
 * exact fp16 in this workspace (M * K * 2 bytes), so that every output tile
 * streams them with TMA instead of converting them again. For W4_OP_W4A8 the
 * figure also depends on N and the group: when the M x N output tiles would
 * fill the GPU's SMs poorly, the GEMM splits K, and the workspace then also
 * holds the parts' fp32 partial sums after the widened activations. Either
 * every tile is split into up to 4 parts (parts * M * N * 4 bytes), or, when
 * only the last wave of tiles is at most half full, each of that wave's r
 * tiles is split into up to 16 parts (r * parts * 128 * 256 * 4 bytes). A W4A8
 * workspace of only M * K * 2 bytes is still accepted; the GEMM then runs
 * unsplit. The caller allocates
 * the workspace (16-byte aligned); its contents on entry do not matter and
 * are overwritten.
 */
size_t w4_workspace_bytes(int32_t op, int64_t M, int64_t N, int64_t K, int32_t group);

/*
 * Dynamic per-token symmetric activation quantization.
 * [INC] apply_weights (dynamic_per_token_int8_quant_ref(x, True, 8): per-token,
 * symmetric, 8 bits) for int8; [FP8] W4AFP8Config.__init__ (input_quant: 8-bit
 * float, symmetric, per token, dynamic) for e4m3.
 *
 *   x      [M, K] bf16 or fp16 (x_dtype W4_BF16 / W4_FP16; [INC] class
 *          docstring: the activations may be bf16 or fp16)
 *   q      [M, K] int8 (q_dtype W4_INT8) or e4m3fn codes (q_dtype W4_FP8_E4M3)
 *   scale  [M] fp32
 * Per row: amax = max_k |x|; s = amax / Q in fp32 with Q = 127 (int8) or 448
 * (e4m3); s = 1 when amax == 0.  int8: q = clamp(rne(x / s), -127, 127).
 * e4m3: q = e4m3(x / s), round to nearest even, saturating at +-448. The
 * divide is the IEEE fp32 divide. Errors: NULL, ALIGN (K % 8), DTYPE, SHAPE.
 */
w4_status w4_quant_act_per_token(const void* x, int32_t x_dtype, int64_t M, int64_t K,
                                 int32_t q_dtype, void* q, float* scale, void* stream);

/*
 * W4A8 linear: int8 activations x int4 GPTQ weights, fp16 group scales.
 * [INC] apply_weights (int4_gemm_w4a8(quant_x, x_scale, ..., qweight,
 * scales_fp16, ..., group_size, ..., bias)) and the class docstring (both scale
 * tensors are read as fp16; bf16 scales are rejected, not misread).
 *
 *   qx       [M, K] int8            (from w4_quant_act_per_token)
 *   x_scale  [M] fp32
 *   qweight  [K/8, N] int32, GPTQ "NT": nibble j (bits 4j..4j+3) of word
 *            [i, n] is the code of input column 8i+j, output n
 *   w_scale  [G, N] fp16 with G = K/group (G = 1 for group -1); w_scale_dtype
 *            must be W4_FP16
 *   bias     [N] bf16 or NULL
 *   y        [M, N] bf16
 * y[m,n] = bf16( x_scale[m] * sum_g w_scale[g,n] * P[m,g,n] + bias[n] ), with
 * P[m,g,n] = sum_{k in g} qx[m,k] * (q[k,n] - 8) formed exactly in integers
 * and the group scale applied in fp32. group: -1 or a multiple of 16 dividing
 * K (else UNSUPPORTED); K % 16 == 0. workspace: at least
 * w4_workspace_bytes(W4_OP_W4A8, M, N, K, group) bytes (W4_ERR_WORKSPACE).
 */
w4_status w4a8_gemm(const void* qx, const float* x_scale, const void* qweight,
                    const void* w_scale, int32_t w_scale_dtype, int32_t group,
                    const void* bias, void* y, int64_t M, int64_t N, int64_t K,
                    void* workspace, size_t workspace_bytes, void* stream);

/*
 * w4a8_gemm for callers that cannot allocate device memory (no counterpart on
 * the source pages: a service of this library). Same arguments and results as
 * w4a8_gemm, minus the workspace: it uses a 32 MiB workspace built into the
 * library, a device array that every GPU which loads the library holds until
 * the process exits. It allocates nothing itself.
 *   - M * K must be at most 16,777,216 (2 bytes of workspace per activation),
 *     else W4_ERR_UNSUPPORTED with a message in w4_last_error().
 *   - The array's device address is looked up on the current device, the
 *     first time the entry point runs in a CUDA context and again whenever the
 *     current context changes (after a device reset, for instance); make the
 *     first call on a device before any stream capture. The stream must belong
 *     to the current device, else W4_ERR_CUDA.
 *   - Every call shares the one array and overwrites it: calls whose kernels
 *     may overlap on the GPU (other streams, other host threads) race and
 *     must be serialized by the caller. Nothing in the array needs to start
 *     at zero; it keeps the last call's contents.
 */
w4_status w4a8_gemm_noalloc(const void* qx, const float* x_scale, const void* qweight,
                            const void* w_scale, int32_t w_scale_dtype, int32_t group,
                            const void* bias, void* y, int64_t M, int64_t N, int64_t K, void* stream);

/*
 * The integer group partials of w4a8_gemm, from the same tensor-core path:
 *   partials [M, G, N] int32, P[m,g,n] = sum_{k in g} qx[m,k] * (q[k,n] - 8).
 * Same argument rules as w4a8_gemm. Meant for verifying the integer core;
 * group (or K for -1) must be at most 16384 so that |P| <= 127 * 8 * group
 * stays below 2^24.
 */
w4_status w4a8_group_partials(const void* qx, const void* qweight, int32_t group,
                              int32_t* partials, int64_t M, int64_t N, int64_t K,
                              void* workspace, size_t workspace_bytes, void* stream);

/*
 * W4A8 linear from bf16 activations: w4_quant_act_per_token (int8) fused into
 * the GEMM's activation pass, so the int8 codes never go to memory: each row
 * is quantized exactly as w4_quant_act_per_token does ([INC] apply_weights:
 * per-token symmetric int8 right before the GEMM) and its codes are written
 * straight into the workspace as the exact fp16 operands of the tensor-core
 * kernel; then y is computed as by w4a8_gemm.
 *
 *   x        [M, K] bf16, 16-byte aligned
 *   x_scale  [M] float32, written (the per-token scales the GEMM used)
 *   other arguments, limits and errors as w4a8_gemm; workspace: at least
 *   w4_workspace_bytes(W4_OP_W4A8, M, N, K, group) bytes.
 * y equals w4a8_gemm applied to w4_quant_act_per_token(x) bit for bit.
 */
w4_status w4a8_gemm_bf16in(const void* x, const void* qweight, const void* w_scale, int32_t w_scale_dtype,
                           int32_t group, const void* bias, void* y, float* x_scale, int64_t M, int64_t N, int64_t K,
                           void* workspace, size_t workspace_bytes, void* stream);

/*
 * W4A16 linear for decode: bf16 activations x the same GPTQ qweight
 * ([INC] class docstring: int4_gemm_w4a16 reads bit-identical weights) with
 * fp16 or bf16 group scales and optional bf16 additive zeros
 * ([OMNI] module docstring: w = (q - 8) * scale + zero).
 *
 *   x        [M, K] bf16
 *   qweight  [K/8, N] int32 GPTQ (as in w4a8_gemm)
 *   w_scale  [G, N], w_scale_dtype W4_FP16 or W4_BF16, 16-byte aligned
 *   zeros    [G, N] bf16 or NULL (symmetric), 16-byte aligned
 *   bias     [N] bf16 or NULL
 *   y        [M, N] bf16
 * y[m,n] = bf16( sum_g [ s[g,n] * sum_{k in g} x[m,k] (q[k,n]-8)
 *                        + z[g,n] * sum_{k in g} x[m,k] ] + bias[n] ),
 * products exact, sums in fp32. Built for small M (tokens are processed in
 * blocks of up to 8, each block one pass over the weights, its x held in
 * shared memory); group: -1 or a multiple of 64 dividing K; K % 64 == 0 and
 * one token row of x must fit in shared memory (K up to about 64000), else
 * W4_ERR_UNSUPPORTED.
 * Launched with programmatic dependent launch: the kernel may start, and
 * start streaming qweight with its scales and zeros, while the kernel before
 * it on `stream` is still finishing (it waits for that kernel before it reads
 * x or the bias, or writes y). So qweight, w_scale and zeros must not be
 * written by a kernel that signals its dependents early, unless a kernel that
 * does not, or a synchronization, stands between the two on the stream (one
 * early signaller after another lets this kernel start while the first still
 * runs). Early signallers are this kernel, those of the fp8 block-scaled
 * layer and its grouped router, those of the 4-bit floating point products and those of
 * w4_moe_decode; every other kernel of this library, and ordinary library kernels, are waited
 * for in full.
 */
w4_status w4a16_gemm(const void* x, const void* qweight, const void* w_scale, int32_t w_scale_dtype,
                     const void* zeros, int32_t group, const void* bias, void* y,
                     int64_t M, int64_t N, int64_t K, void* stream);

/*
 * w4a16_gemm from and to host memory, for a caller whose activations and
 * results live on the host: one call queues on `stream` the copy of x_host
 * [M, K] bf16 into x_dev, the w4a16_gemm of x_dev into y_dev, and the copy of
 * y_dev [M, N] into y_host. x_dev and y_dev are caller-owned device buffers
 * (16- and 8-byte aligned) and hold x and y afterwards. When x_host and y_host
 * are both page-locked (x_host 16-byte aligned) no copy-engine job is queued:
 * the call's L2-prefetch grid copies x_host into x_dev and the GEMV writes
 * y_host along with y_dev, so consecutive calls on a stream overlap as
 * device-only calls do; otherwise each copy is one cudaMemcpyAsync,
 * asynchronous only for page-locked memory. y_host holds
 * the result once `stream` has been synchronized; x_host and y_host must not
 * be touched by the host until then. Other arguments and errors as
 * w4a16_gemm; nothing is queued when validation fails.
 */
w4_status w4a16_gemm_host(const void* x_host, void* x_dev, const void* qweight, const void* w_scale,
                          int32_t w_scale_dtype, const void* zeros, int32_t group, const void* bias, void* y_dev,
                          void* y_host, int64_t M, int64_t N, int64_t K, void* stream);

/*
 * W4AFP8 grouped expert linear ([FP8] W4AFP8Config: int4 group-128 routed
 * experts, symmetric, fp8 per-token dynamic activations; get_checkpoint_weight_mapper:
 * compressed-tensors "weight_packed" / "weight_scale" layout).
 *
 *   qx              [R, K] e4m3fn codes, rows grouped by expert
 *   x_scale         [R] fp32
 *   expert_offsets  DEVICE int32 [E+1]: rows of expert e are
 *                   [offsets[e], offsets[e+1]); offsets[0] = 0, offsets[E] = R,
 *                   non-decreasing (an expert may own no rows)
 *   qweight         [E, N, K/8] int32: nibble j of word [e, n, i] is the code
 *                   of input column 8i+j of output n of expert e
 *   w_scale         [E, N, K/group] fp16 (w_scale_dtype W4_FP16)
 *   y               [R, N] bf16
 * y[r,n] = bf16( x_scale[r] * sum_g w_scale[e,n,g] * sum_{k in g} x[r,k] (q[e,n,k]-8) )
 * with e the expert owning row r. group: a multiple of 16 dividing K, or -1;
 * K % 32 == 0. workspace: at least w4_workspace_bytes(W4_OP_W4AFP8_MOE, R, N, K,
 * group) bytes. Offsets are not validated on the host (they live on the device);
 * rows outside [0, R) are never written.
 */
w4_status w4afp8_moe_grouped_gemm(const void* qx, const float* x_scale, const int32_t* expert_offsets,
                                  int32_t E, const void* qweight, const void* w_scale,
                                  int32_t w_scale_dtype, int32_t group, void* y,
                                  int64_t R, int64_t N, int64_t K,
                                  void* workspace, size_t workspace_bytes, void* stream);

/*
 * The routed MoE layer around w4afp8_moe_grouped_gemm. [FP8] (module
 * docstring, W4AFP8Config.get_quant_method) gives int4 routed experts with
 * fp8 per-token activations but prints no routing or activation formula; the
 * plain top-k layer is taken:
 *   route:    per token the k experts with the largest logits, equal logits
 *             in ascending expert order; weight = softmax probability over
 *             all E experts (fp32), or divided by the sum over the k chosen
 *             when renormalize != 0;
 *   rows:     the T*k pairs (token, choice) listed by expert, then token;
 *   between:  act = bf16(silu(gate) * up) in fp32, gate = columns [0, I) of the
 *             gate_up output, up = [I, 2I); act quantized per row to e4m3
 *             exactly as w4_quant_act_per_token does;
 *   combine:  out[t] = bf16(sum_j w[t, j] * y[row_of[t, j]]), fp32, j ascending.
 * A layer is: w4_moe_route; w4afp8_moe_gemm_bf16in (gate_up, gathering the
 * token rows); w4_moe_silu_mul_quant_fp8; w4afp8_moe_grouped_gemm (down);
 * w4_moe_combine.
 */

/*
 * w4_moe_route: logits [T, E], bf16 (logits_f32 == 0) or fp32 (logits_f32
 * != 0); 1 <= E <= 1024, 1 <= top_k <= min(E, 64). Outputs, device buffers
 * owned by the caller:
 *   topk_ids      int32 [T, top_k]  chosen experts, largest logit first
 *   topk_weights  fp32  [T, top_k]  weights
 *   offsets       int32 [E+1]       expert e owns rows [offsets[e], offsets[e+1])
 *   row_token     int32 [T*top_k]   token of each row
 *   row_of        int32 [T, top_k]  row of each (token, choice)
 * workspace: at least w4_workspace_bytes(W4_OP_MOE_ROUTE, T, E, 1, 0) bytes,
 * 4-byte aligned. NaN logits are outside the contract (they are taken as
 * -inf). T == 0 launches nothing and returns W4_OK.
 */
w4_status w4_moe_route(const void* logits, int32_t logits_f32, int64_t T, int32_t E, int32_t top_k,
                       int32_t renormalize, int32_t* topk_ids, float* topk_weights, int32_t* offsets,
                       int32_t* row_token, int32_t* row_of, void* workspace, size_t workspace_bytes,
                       void* stream);

/*
 * w4_moe_gather_quant_fp8: row r of q/scale is token row_token[r] of x
 * [T, K] bf16 quantized per row to e4m3 (the codes and scale that
 * w4_quant_act_per_token gives that row). q [R, K] (x and q 16-byte aligned),
 * scale [R] fp32, K % 8 == 0. A row_token entry outside [0, T) gives a zero row
 * with scale 1 and sets W4_ERR_SHAPE in the device status word
 * (w4_device_status).
 */
w4_status w4_moe_gather_quant_fp8(const void* x, int64_t T, int64_t K, const int32_t* row_token, int64_t R,
                                  void* q, float* scale, void* stream);

/*
 * w4afp8_moe_gemm_bf16in: w4_moe_gather_quant_fp8 fused into
 * w4afp8_moe_grouped_gemm. The gathered rows are quantized straight into the
 * GEMM's workspace (no fp8 copy in HBM); x_scale [R] receives the row scales.
 * row_token may be NULL (then R must equal T and row r is token r). y equals
 * w4afp8_moe_grouped_gemm applied to w4_moe_gather_quant_fp8(x) bit for bit.
 * Other arguments and limits as w4afp8_moe_grouped_gemm.
 */
w4_status w4afp8_moe_gemm_bf16in(const void* x, int64_t T, const int32_t* row_token, const int32_t* expert_offsets,
                                 int32_t E, const void* qweight, const void* w_scale, int32_t w_scale_dtype,
                                 int32_t group, void* y, float* x_scale, int64_t R, int64_t N, int64_t K,
                                 void* workspace, size_t workspace_bytes, void* stream);

/*
 * w4_moe_silu_mul_quant_fp8: h [R, 2I] bf16 (the gate_up output) -> q [R, I]
 * e4m3 codes and scale [R] fp32; act [R, I] bf16 receives the activations
 * before quantization when not NULL. I % 8 == 0; h, q and act 16-byte aligned.
 */
w4_status w4_moe_silu_mul_quant_fp8(const void* h, int64_t R, int64_t I, void* q, float* scale, void* act,
                                    void* stream);

/*
 * w4_moe_combine: y [R, H] bf16 (the down output, expert-sorted rows),
 * topk_weights [T, top_k] fp32 and row_of [T, top_k] int32 from w4_moe_route;
 * out [T, H] bf16. H % 8 == 0; y and out 16-byte aligned. A row_of entry
 * outside [0, R) adds nothing and sets W4_ERR_SHAPE in the device status word.
 */
w4_status w4_moe_combine(const void* y, int64_t R, int64_t H, const float* topk_weights, const int32_t* row_of,
                         int64_t T, int32_t top_k, void* out, void* stream);

/*
 * w4_moe_route_grouped: routing with sigmoid or softmax scores, a balance bias
 * and expert groups. Outputs and their layouts as w4_moe_route, so every expert
 * entry point takes its row order. workspace: at least w4_workspace_bytes(
 * W4_OP_MOE_ROUTE_GROUPED, T, E, 1, 0) bytes, 4-byte aligned (0 bytes for few
 * tokens: it may then be NULL).
 *
 *   score[e]  sigmoid(logit) or softmax over all E experts (scoring)
 *   key[e]    what the choice goes by: the logit itself (bias NULL), or
 *             fl(score[e] + bias[e]) with bias fp32 [E]
 *   groups    E / n_group consecutive experts each; a group's value is its
 *             largest key (bias NULL), or the sum of its two largest keys (of
 *             its one key, for groups of one). The topk_group best groups stay
 *             open, equal values in ascending group order.
 *   choice    the top_k largest keys of the open groups, largest first, equal
 *             keys in ascending expert order
 *   weight    score (without the bias), divided by the sum of the chosen
 *             scores when renormalize != 0, times scale
 * All in fp32. The steps a choice depends on are fixed: sigmoid is
 * fl(1 / fl(1 + exp(-l))), and with a bias the softmax denominator is summed in
 * fp64 and rounded once.
 *
 * 1 <= E <= 1024; n_group divides E (W4_ERR_GROUP), at most 32
 * (W4_ERR_UNSUPPORTED); 1 <= topk_group <= n_group; 1 <= top_k <= min(64,
 * topk_group * E / n_group). A logit of -inf scores 0. Without a bias its key is
 * -inf, so that it is chosen only when nothing else is open; with one its key is
 * bias[e], which can beat another expert's (a bias of -inf closes an expert there).
 * Where the chosen scores sum to 0, as in a row that is masked altogether,
 * renormalized weights are 0. NaN logits count as -inf, +inf as the largest finite
 * fp32; bias must not be NaN. T == 0 launches nothing.
 */
w4_status w4_moe_route_grouped(const void* logits, int32_t logits_f32, const float* bias, int64_t T, int32_t E,
                               int32_t top_k, int32_t n_group, int32_t topk_group, int32_t scoring,
                               int32_t renormalize, float scale, int32_t* topk_ids, float* topk_weights,
                               int32_t* offsets, int32_t* row_token, int32_t* row_of, void* workspace,
                               size_t workspace_bytes, void* stream);

/*
 * The fp8 block-scaled layer: e4m3 weights with one fp32 scale per 128 x 128
 * block, e4m3 activations with one fp32 scale per token and 128 columns. [FP8]
 * (W4AFP8Config) keeps every layer of the checkpoint but the routed experts in
 * this form ("weight" e4m3 [N, K], "weight_scale_inv" [ceil(N/128),
 * ceil(K/128)], dynamic activations); checkpoints whose experts were not
 * converted to int4 keep those in it too.
 *
 * The entry points of this layer are launched with programmatic dependent launch,
 * as w4a16_gemm is, and signal their own dependents early. They may start
 * streaming qweight while the kernels before them on `stream` are finishing and wait
 * for those before they touch anything else. So qweight must not be written by a
 * kernel that signals its dependents early (any of this layer, or w4a16_gemm), unless
 * a kernel that does not, or a synchronization, stands between the two on the stream.
 *
 * w4_quant_act_per_block: per row and block of 128 columns (the last one may be
 * shorter) amax = max |x|, s = amax / 448 in fp32 (1 where that is 0),
 * q = e4m3(fl(x / s)), round to nearest even, saturating; the divides are IEEE, and
 * zeros keep their sign. NaN counts for nothing in amax and has a NaN code (a block of
 * NaN alone a NaN scale); an infinity makes its block's scale infinite, its own code
 * NaN and the block's other codes 0.
 *   x [M, K] bf16 or fp16 (x_dtype), 16-byte aligned; K % 8 == 0
 *   q [M, K] e4m3 codes, 16-byte aligned; scale [M, ceil(K/128)] fp32
 */
w4_status w4_quant_act_per_block(const void* x, int32_t x_dtype, int64_t M, int64_t K, void* q, float* scale,
                                 void* stream);

/*
 * w4_silu_mul_quant_block: h [R, 2I] bf16 (gate columns first) -> the codes and
 * scales of silu(gate) * up, quantized as by w4_quant_act_per_block. The product
 * stays in fp32 up to its rounding to e4m3. It is within a few fp32 ulp of the
 * definition as far as fp32 reaches (a gate of -100 times a large up is not 0), of a
 * gate below -64 within 8. A gate of +inf gives an infinite product, -inf NaN.
 * q [R, I], scale [R, ceil(I/128)]; I % 8 == 0; h and q 16-byte aligned.
 */
w4_status w4_silu_mul_quant_block(const void* h, int64_t R, int64_t I, void* q, float* scale, void* stream);

/*
 * w4_fp8_block_gemm:
 *   y[m, n] = bf16( sum_b x_scale[m, b] * w_scale[n / 128, b] * P[m, b, n] + bias[n] ),
 *   P[m, b, n] = sum over the 128 columns k of block b of qx[m, k] * qweight[n, k],
 * everything after the e4m3 codes in fp32.
 *   qx       [M, K] e4m3 codes        x_scale [M, ceil(K/128)] fp32
 *   qweight  [N, K] e4m3 codes        w_scale [ceil(N/128), ceil(K/128)] fp32
 *   bias     [N] bf16 or NULL         y       [M, N] bf16
 * N % 8 == 0, K % 16 == 0 (a K that is a multiple of 8 only: W4_ERR_UNSUPPORTED);
 * neither has to be a multiple of 128. Matrices and the bias are 16-byte aligned. Few
 * rows take a form that streams the weights once for all of them; M == 1 is
 * the decode call. Sums are taken in a fixed order: a call's outputs are the same
 * every time. workspace: w4_workspace_bytes(W4_OP_FP8_BLOCK, M, N, K, 0) bytes,
 * 16-byte aligned, for the fp32 sums of tiles that are split along K (0 bytes
 * where none is). NULL, or a smaller one: no tile is split.
 */
w4_status w4_fp8_block_gemm(const void* qx, const float* x_scale, const void* qweight, const float* w_scale,
                            const void* bias, void* y, int64_t M, int64_t N, int64_t K, void* workspace,
                            size_t workspace_bytes, void* stream);

/*
 * w4_fp8_block_gemm_bf16in: w4_quant_act_per_block and w4_fp8_block_gemm in one
 * call: x [M, K] bf16 or fp16 (x_dtype), its codes and scales in the workspace
 * (at least w4_workspace_bytes(W4_OP_FP8_BLOCK_IN, M, N, K, 0) bytes, 16-byte
 * aligned; 0 bytes for few rows, where the product quantizes x itself and the
 * workspace may be NULL; with only M * K + 4 * M * ceil(K/128) bytes, rounded up
 * to 16, no tile is split). y equals the two calls' with their workspaces bit for
 * bit. The product's weights start streaming while x is being quantized.
 */
w4_status w4_fp8_block_gemm_bf16in(const void* x, int32_t x_dtype, const void* qweight, const float* w_scale,
                                   const void* bias, void* y, int64_t M, int64_t N, int64_t K, void* workspace,
                                   size_t workspace_bytes, void* stream);

/*
 * w4_fp8_block_moe_grouped_gemm: the same product over expert-sorted rows, as
 * w4afp8_moe_grouped_gemm takes them: rows [offsets[e], offsets[e+1]) of qx
 * [R, K] times expert e of qweight [E, N, K], w_scale [E, ceil(N/128),
 * ceil(K/128)] fp32; y [R, N] bf16. 1 <= E <= 1024. Offsets live on the device
 * and are not validated; rows outside [0, R) are neither read nor written.
 */
w4_status w4_fp8_block_moe_grouped_gemm(const void* qx, const float* x_scale, const int32_t* expert_offsets, int32_t E,
                                        const void* qweight, const float* w_scale, void* y, int64_t R, int64_t N,
                                        int64_t K, void* stream);

/*
 * w4_fp8_block_moe_gemm_bf16in: row r is token row_token[r] of x [T, K] bf16
 * (row_token NULL: R == T and row r is token r), quantized per block into the
 * workspace (w4_workspace_bytes(W4_OP_FP8_BLOCK_IN, R, N, K, E) bytes; with only
 * R * K + 4 * R * ceil(K/128) bytes, rounded up to 16, a token is quantized again for
 * each of its rows), then w4_fp8_block_moe_grouped_gemm. A row_token entry outside [0, T) gives a
 * zero row and sets W4_ERR_SHAPE in the device status word.
 */
w4_status w4_fp8_block_moe_gemm_bf16in(const void* x, int64_t T, const int32_t* row_token, const int32_t* expert_offsets,
                                       int32_t E, const void* qweight, const float* w_scale, void* y, int64_t R,
                                       int64_t N, int64_t K, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Microscaled 4-bit floating point (no counterpart on the source pages). Codes are
 * e2m1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and, with the high bit, their negatives; two codes a byte,
 * the lower column in the low half. Every row has a scale per block of columns, in
 * row-major order, as checkpoints hold them:
 *     W4_FMT_MXFP4: blocks of 32, scale 2^(byte - 127) (e8m0; 255 is NaN);
 *     W4_FMT_NVFP4: blocks of 16, scale e4m3 times an fp32 scale of the whole
 *                   tensor, which is a device scalar (`global`; NULL: 1; must be NULL
 *                   for mxfp4, else W4_ERR_UNSUPPORTED). No block scale is negative.
 *
 * w4_quant_fp4: x [M, K] bf16 or fp16 to codes q [M, K/2] bytes and scale [M, K/32]
 * (mxfp4) or [M, K/16] (nvfp4) bytes, activations or weights alike. With amax
 * the block's largest magnitude, every step in fp32 with IEEE rounding:
 *     mxfp4: e = clamp(floor(log2 amax) - 2, -127, 127) (-127 for a block of zeros),
 *            q = e2m1(x 2^-e);
 *     nvfp4: s = e4m3(fl(fl(amax / 6) / global)), d = fl(s global), q = e2m1(fl(x / d)), 0 where d = 0;
 * e2m1 and e4m3 round to nearest even and hold at the largest magnitude (6, 448). A
 * block that holds a NaN or an infinity gets a NaN scale and codes 0, so that the row of
 * a product is NaN. global must be positive and finite. K % 32 == 0 (W4_ERR_UNSUPPORTED
 * for other multiples of 8); x and q 16-byte aligned, global 4-byte.
 *
 * w4_silu_mul_quant_fp4: the same of fl(fl(g / fl(1 + expf(-g))) u) for h [R, 2I] bf16, g its
 * first I columns and u the others; I % 32 == 0.
 *
 * w4_dequant_fp4: out [M, K] (out_dtype W4_BF16 or W4_FP16) = code times scale (nvfp4: times
 * fl(scale global)) in fp32, rounded once.
 */
w4_status w4_quant_fp4(const void* x, int32_t x_dtype, int32_t format, const float* global, int64_t M, int64_t K,
                       void* q, void* scale, void* stream);
w4_status w4_silu_mul_quant_fp4(const void* h, int32_t format, const float* global, int64_t R, int64_t I, void* q,
                                void* scale, void* stream);
w4_status w4_dequant_fp4(const void* q, const void* scale, int32_t format, const float* global, int64_t M, int64_t K,
                         int32_t out_dtype, void* out, void* stream);

/*
 * w4_fp4_gemm: both operands in the same 4-bit format,
 *     y[m, n] = bf16( x_global w_global sum_b x_scale[m, b] w_scale[n, b] sum_{k in b} qx[m, k] qw[n, k] + bias[n] ),
 * products exact, sums in fp32 on the tensor cores.
 *   qx       [M, K/2] bytes, x_scale [M, K/32 or K/16] bytes
 *   qweight  [N, K/2] bytes, w_scale [N, K/32 or K/16] bytes
 *   x_global, w_global  device fp32 scalars (nvfp4) or NULL
 *   bias     [N] bf16 or NULL         y       [M, N] bf16
 * N % 8 == 0; rows of scales are whole 32-bit words: K % 128 == 0 (mxfp4) or K % 64 == 0
 * (nvfp4), else W4_ERR_UNSUPPORTED. Matrices and the bias are 16-byte aligned, scales
 * 4-byte. Few rows take a form that streams the weights once; M == 1 is the decode call.
 * Sums are taken in a fixed order: a call's outputs are the same every time.
 *
 * w4_fp4_gemm_bf16in: x [M, K] bf16 or fp16, quantized as w4_quant_fp4 does into the
 * workspace (at least w4_workspace_bytes(W4_OP_FP4_IN, M, N, K, 16 or 32) bytes, 16-byte
 * aligned; 0 bytes for few rows, where the product quantizes x itself and the
 * workspace may be NULL), then w4_fp4_gemm; y equals the two calls' bit for bit.
 *
 * w4_fp4_moe_grouped_gemm: the product over expert-sorted rows, as
 * w4afp8_moe_grouped_gemm takes them: rows [offsets[e], offsets[e+1]) of qx [R, K/2] times
 * expert e of qweight [E, N, K/2], w_scale [E, N, K/32 or K/16]; w_global [E] or NULL; y [R, N]
 * bf16. 1 <= E <= 1024. Offsets live on the device and are not validated; rows outside
 * [0, R) and rows of no expert are not written.
 *
 * w4_fp4_moe_gemm_bf16in: row r is token row_token[r] of x [T, K] bf16 (row_token NULL: R
 * == T and row r is token r), quantized into the workspace
 * (w4_workspace_bytes(W4_OP_FP4_MOE_IN, R, N, K, 16 or 32) bytes; with only those of
 * W4_OP_FP4_IN a token is quantized again for each of its rows), then
 * w4_fp4_moe_grouped_gemm. A row_token entry outside [0, T) gives a zero row and sets
 * W4_ERR_SHAPE in the device status word.
 *
 * The products are launched as programmatic dependents that start streaming weights and
 * their scales early, and let their own dependents go early, as w4a16_gemm does; the rule
 * given there for what may write weights holds for qweight, w_scale and w_global too.
 * The quantizers above are waited for in full, so a weight may be quantized right before.
 */
w4_status w4_fp4_gemm(const void* qx, const void* x_scale, const float* x_global, const void* qweight,
                      const void* w_scale, const float* w_global, int32_t format, const void* bias, void* y, int64_t M,
                      int64_t N, int64_t K, void* stream);
w4_status w4_fp4_gemm_bf16in(const void* x, int32_t x_dtype, const float* x_global, const void* qweight,
                             const void* w_scale, const float* w_global, int32_t format, const void* bias, void* y,
                             int64_t M, int64_t N, int64_t K, void* workspace, size_t workspace_bytes, void* stream);
w4_status w4_fp4_moe_grouped_gemm(const void* qx, const void* x_scale, const float* x_global,
                                  const int32_t* expert_offsets, int32_t E, const void* qweight, const void* w_scale,
                                  const float* w_global, int32_t format, void* y, int64_t R, int64_t N, int64_t K,
                                  void* stream);
w4_status w4_fp4_moe_gemm_bf16in(const void* x, int64_t T, const float* x_global, const int32_t* row_token,
                                 const int32_t* expert_offsets, int32_t E, const void* qweight, const void* w_scale,
                                 const float* w_global, int32_t format, void* y, int64_t R, int64_t N, int64_t K,
                                 void* workspace, size_t workspace_bytes, void* stream);

/*
 * w4_moe_decode: a whole routed MoE layer for a few tokens, in two kernels. From x [T, H]
 * bf16 and router logits [T, E] (bf16, or fp32 where logits_f32 != 0),
 *     experts e and weights w of token t as w4_moe_route_grouped gives them (bias,
 *     top_k, n_group, topk_group, scoring, renormalize, scale as there);
 *     h = gate_up[e] x_t;  a = silu(h[0 .. I)) h[I .. 2I);  y_t = bf16( sum_e w down[e] a ).
 * Activations stay 16-bit (the W4A16 form of the experts); sums are fp32. x is taken as
 * fp16 times a power of two per token (a bf16 loses nothing down to 2^-29 of the token's largest
 * number) and a to 22 bits (two fp16 numbers with an exponent per eight columns), down to 2^-29 of the
 * largest among 128 columns. A token that holds a NaN or an infinity gives no finite numbers and leaves the
 * others alone. Outputs are the same every time.
 *   format   W4_FMT_INT4: gate_up [E, 2I, H/8] int32, gate_up_scale [E, 2I, H/group] fp16
 *            (the layout of w4afp8_moe_grouped_gemm); group: gate_up_group and
 *            down_group, multiples of 32 that divide H and I, or -1;
 *            W4_FMT_MXFP4, W4_FMT_NVFP4: gate_up [E, 2I, H/2] bytes, gate_up_scale [E, 2I,
 *            H/32 or H/16] bytes as w4_quant_fp4 gives them (groups ignored)
 *   gate_up_global, down_global  fp32 [E] (nvfp4) or NULL
 *   down     [E, H, I/8] int32 or [E, H, I/2] bytes, down_scale alike
 *   y        [T, H] bf16
 * Limits (W4_ERR_UNSUPPORTED): T <= 16, E <= 256, top_k <= 32, H and I multiples of 64, and
 * shared memory for T rows of x beside the copies in flight: with I up to 7168, 16 tokens fit at H
 * up to 2560 and 7 at H = 4096; int4 groups of 128 leave room for more. Where rows of scales can be copied 512
 * columns at a time (H and I multiples of 512 in mxfp4, of 256 in nvfp4 and int4 groups of 32, of 512 in groups of 64), 14 fit
 * at H = 4096 and 8 at H = 7168, whatever I. For more tokens w4_moe_route_grouped and the grouped products.
 * In int4 it takes a third to a quarter of these calls' time at any number of tokens. In the 4-bit floating point
 * formats those, whose activations have 4 bits, are faster from some 50 MB of chosen experts' weights on (64 experts of
 * 2048 x 1408, 8 chosen, mxfp4: 1 token 24 us and 29, 2 34 and 32, 16 100 and 60; 96 of 1024 x 704, 6 chosen, nvfp4: 8 tokens
 * 32 and 34, 16 47 and 37).
 * Matrices, scales and the workspace are 16-byte aligned. workspace: at least
 * w4_workspace_bytes(W4_OP_MOE_DECODE, T, top_k, I, 0) bytes. x, logits, bias and weights are
 * read after the kernels before are done; its own dependents may start early, as those
 * of w4a16_gemm.
 */
w4_status w4_moe_decode(const void* x, const void* logits, int32_t logits_f32, const float* bias, int64_t T, int32_t E,
                        int32_t top_k, int32_t n_group, int32_t topk_group, int32_t scoring, int32_t renormalize,
                        float scale, int32_t format, const void* gate_up, const void* gate_up_scale,
                        const float* gate_up_global, int32_t gate_up_group, const void* down, const void* down_scale,
                        const float* down_global, int32_t down_group, void* y, int64_t H, int64_t I, void* workspace,
                        size_t workspace_bytes, void* stream);

/*
 * Weight-side tools (load time, not on the per-token path).
 *
 * w4_quantize_groupwise: the asymmetric min/max 4-bit group quantizer of
 * [OMNI] quantize_groupwise. For each row n of w [N, K] (bf16 or fp16,
 * w_dtype W4_BF16 / W4_FP16) and each group of `group` consecutive columns
 * (group -1 = K), in fp32 with IEEE rounding at every step:
 *     scale = max(max - min, 1e-9) / 15,   zero = min + 8 * scale,
 *     q = clamp(round_half_even((w - min) / scale), 0, 15),
 * so that (q - 8) * scale + zero reproduces the group's extremes. Outputs, all
 * caller-owned device memory:
 *     packed [N, K/2] uint8, two codes per byte, low nibble first
 *            ([OMNI] pack_nibbles: byte j = q[2j] | q[2j+1] << 4)
 *     scale  [N, K/group] float32
 *     zero   [N, K/group] float32
 * Codes, scales and zeros are bit-exact. Requires K and the group even
 * (W4_ERR_UNSUPPORTED otherwise), the group to divide K (W4_ERR_GROUP), w
 * 4-byte aligned (W4_ERR_ALIGN). N == 0 does nothing. NaN/Inf in w are out of
 * contract.
 */
w4_status w4_quantize_groupwise(const void* w, int32_t w_dtype, int64_t N, int64_t K, int32_t group,
                                void* packed, float* scale, float* zero, void* stream);

/*
 * w4_repack_s4_to_uint4b8: [FP8] _repack_signed_int4_to_uint4b8. Every byte
 * of `src` holds two signed int4 values; the output byte holds the same two
 * values as uint4b8 codes (value + 8, so the weight is q - 8), which is XOR
 * 0x88 on the byte. Read as int32, 8 codes per word in the same nibble order.
 * n_bytes may be any size; src and dst must be 16-byte aligned and may be the
 * same buffer (in place); both are caller-owned device memory. Bit-exact.
 */
w4_status w4_repack_s4_to_uint4b8(const void* src, void* dst, int64_t n_bytes, void* stream);

/*
 * Quantized embedding table used as the vocabulary lookup and as the tied
 * output head ([OMNI] CPUInt4EmbeddingMethod: class docstring, embedding,
 * tie_weights). The table is the output of w4_quantize_groupwise, kept row
 * major and shared by both calls:
 *     table  [V, D/2] uint8, two codes per byte, low nibble first
 *     scale  [V, D/group] float32,  zero [V, D/group] float32
 * group -1 means D. D and the group must be multiples of 8 (W4_ERR_ALIGN).
 *
 * w4_embedding_gather: out[t, :] = bf16((q[ids[t], :] - 8) * scale + zero),
 * each fp32 step rounded as the page's fp32 code does (bit-exact). ids: [T]
 * int32 device array; out: [T, D] bf16, 16-byte aligned. An id outside
 * [0, V) gives a row of zeros and records W4_ERR_SHAPE in the device status
 * word (w4_device_status). T == 0 does nothing.
 */
w4_status w4_embedding_gather(const int32_t* ids, int64_t T, const void* table, const float* scale,
                              const float* zero, int64_t V, int64_t D, int32_t group, void* out, void* stream);

/*
 * w4_lm_head_gemv: the tied head for decode, logits y[m, v] =
 * bf16(sum_d h[m, d] * ((q[v, d] - 8) * scale[v, d / group] + zero[v, d / group]))
 * with fp32 accumulation, h [M, D] bf16, y [M, V] bf16, read from the same
 * table (16-byte aligned). Built for small M (tokens in blocks of 8, each one
 * pass over the table); D % 32 == 0, and D <= 8192 when D and the group are
 * multiples of 128 (tensor-core form), else D <= 5792 (8 rows of h in shared
 * memory), otherwise W4_ERR_UNSUPPORTED. M == 0 does nothing.
 */
w4_status w4_lm_head_gemv(const void* h, int64_t M, const void* table, const float* scale, const float* zero,
                          int64_t V, int64_t D, int32_t group, void* y, void* stream);

/* Message for the last non-OK status returned to the calling thread ("" if none). */
const char* w4_last_error(void);

/* Name of a status code. */
const char* w4_status_string(int32_t status);

/*
 * Synchronizes `stream`, then reads and clears the device status word that the
 * pipelined kernels set when a bounded wait runs out. Returns W4_OK,
 * W4_ERR_TIMEOUT, or W4_ERR_CUDA if the synchronize itself failed.
 */
w4_status w4_device_status(void* stream);

/*
 * Self-test of the bounded-wait machinery: launches one CTA that waits on an
 * mbarrier nothing ever arrives at, with a limit of `spin_limit` polls (> 0).
 * The wait runs out, the kernel records W4_ERR_TIMEOUT and returns; a
 * following w4_device_status() returns W4_ERR_TIMEOUT and clears it.
 */
w4_status w4_selftest_bounded_wait(int64_t spin_limit, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* W4_H_ */

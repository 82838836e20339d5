/*
 * awq.h - C ABI of the B200 (sm_100a) AWQ activation-aware scale search and INT4 group quantizer.
 *
 * What the library computes (sources are five web pages about AWQ, cited by title and section):
 *
 *   (1) act_mean[k] = mean_i |X[i,k]|            "显著权重的识别" on the bjdmk.com.cn AWQ article
 *                                                 (S_X(i) = 1/N sum_j |X_ji|); 原理 on the msModelSlim page
 *                                                 "AWQ：激活感知权重量化算法说明" (act_mean = mean(abs(act))).
 *   (2) for ratio_j = j / n_grid, j = 0..n_grid-1 (the grid [0, 1) with step 1/n_grid, 原理 on the
 *       msModelSlim page): s = clamp(act_mean^ratio, min 1e-4); s = s / sqrt(max(s) * min(s)).
 *   (3) W' = W diag(s); asymmetric 4-bit quantization of W' in groups of 128 consecutive in-features:
 *       step = clamp((max - min) / 15, min 1e-5), z = round(-min / step),
 *       q = clamp(round(w' / step) + z, 0, 15), deq = (q - z) * step, w_hat = deq / s
 *       (section 二 of "AWQ 离群激活平滑实操逐通道等价缩放与 4-bit 精度无损转换", gsyq.cn; that page clamps the
 *       step at 1e-8, this library at 1e-5).
 *   (4) loss_j = mean over the N*O outputs of (X W^T - X W_hat_j^T)^2 (the loss L(s) in
 *       "数学等价变换与通道自适应缩放" on the bjdmk.com.cn article; the MSE step of 缩放因子搜索流程 on the
 *       msModelSlim page); the best ratio is the first j reaching the minimum (strict '<' update in the
 *       search loops of both pages).
 *   (5) the INT4 codes of W at the best scales, 8 codes per uint32, plus per-group steps and zeros
 *       (two codes per byte in "GPU 硬件级反量化算子内联融合" on the bjdmk.com.cn article; this library
 *       packs code of in-feature k into word k/8, bits 4*(k%8) .. 4*(k%8)+3).
 *
 * Several linears that read the same input (q/k/v after one norm; NormLinearSubgraph on the msModelSlim
 * page) share one scale vector: pass their weights stacked row-wise as one [O_total, K] matrix.
 *
 * Conventions for every entry point
 *   - Matrices are row-major bfloat16 bit patterns: X is [N, K] (tokens x in-features) with row stride
 *     ldx elements, W is [O, K] (out-features x in-features, torch nn.Linear layout) with row stride ldw.
 *   - Every pointer except those documented as host pointers is a DEVICE pointer of the current CUDA
 *     device. The caller owns all memory; the library never allocates device or host memory.
 *   - Every call is asynchronous on `stream` (NULL selects the legacy default stream) and returns after
 *     validation and enqueueing. A non-OK status means nothing was enqueued, except AWQ_ERR_CUDA from a
 *     failed launch. awq_last_error() then returns a message (thread-local, valid until the next call).
 *   - Pointers must be 16-byte aligned and ldx, ldw multiples of 8 (rows start on 16-byte boundaries).
 *   - group must be 128 (AWQ_ERR_UNSUPPORTED otherwise); K must be a multiple of 128.
 *   - Inputs must be finite; NaN or Inf give unspecified (but memory-safe) results.
 *   - Calls that share a workspace must not overlap on the GPU (serialise them on one stream).
 *   - Device waits inside the kernels are bounded (default 2 s, see awq_set_wait_limit_ns); a wait that
 *     gives up records AWQ_ERR_TIMEOUT in the workspace, makes the remaining kernels of the call skip
 *     their work, and sets *best_j = -1; awq_search_status() reports it.
 */
#ifndef AWQ_B200_H
#define AWQ_B200_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define AWQ_API __attribute__((visibility("default")))
#else
#define AWQ_API
#endif

typedef struct CUstream_st *awq_stream_t; /* identical to cudaStream_t */

typedef enum awq_status {
  AWQ_OK = 0,
  AWQ_ERR_INVALID_ARG = 1, /* null pointer, bad size, misalignment, n_grid out of range */
  AWQ_ERR_UNSUPPORTED = 2, /* group not 128 (0 with AWQ_FLAG_QUANT_INT8), or a device other than sm_100 */
  AWQ_ERR_WORKSPACE = 3,   /* workspace null or smaller than the *_workspace_size() query */
  AWQ_ERR_CUDA = 4,        /* a CUDA runtime call or launch failed; message from the runtime */
  AWQ_ERR_TIMEOUT = 5      /* a bounded device wait gave up (reported by awq_search_status) */
} awq_status;

/* Flags for the *_ex entry points (0 = the production behaviour of the plain entry points). */
#define AWQ_FLAG_EXACT_DIVISION 0x1u /* every w'/step quotient by IEEE division, no reciprocal fast path;
                                        in the search also the unscale w_hat = RN32(deq / s) */
#define AWQ_FLAG_EXACT_POW 0x2u      /* every act_mean^ratio by the double-double path, no fp64 pow */
#define AWQ_FLAG_INJECT_STALL 0x100u /* test hook: the loss GEMM waits on a barrier nobody signals */
/* Candidate-scale rule of the search (default: 原理 on the msModelSlim page, see (2) below). */
#define AWQ_FLAG_SCALES_WEIGHT_AWARE 0x10u /* AWQChannelScaler on the bjdmk.com.cn article: see (2) */
#define AWQ_FLAG_SCALES_RMS 0x20u          /* search_smooth_scaling_factors, gsyq.cn section 二: see (2) */
/* Weight quantizer of the search (default: asymmetric INT4 in groups of 128, see (3)). */
#define AWQ_FLAG_QUANT_INT8 0x40u /* symmetric INT8, one step per output channel: see (5b); group must be 0 */

#define AWQ_MAX_N_GRID 64

/* Message of the last failing call on this thread ("" if none). */
AWQ_API const char *awq_last_error(void);

/* Library ABI version (major * 100 + minor). */
AWQ_API int awq_version(void);

/* Upper bound, in nanoseconds, of every device-side wait (mbarrier waits of the loss GEMM). Default
 * 2e9. Applies to calls enqueued after it. Values below 1e6 are raised to 1e6. */
AWQ_API void awq_set_wait_limit_ns(uint64_t ns);

/* Test hook, like AWQ_FLAG_INJECT_STALL: in later calls of awq_w4a16_experts the MMAs of tile `tile` (tiles counted over the
 * experts of more than 8 rows) wait for a barrier that nobody signals. -1, the default: nowhere. */
AWQ_API void awq_set_experts_stall(int tile);

/* ---------------------------------------------------------------------------------------------------
 * (1) Activation statistic.  act_mean[k] = RN32(RN64(S_k / N)) with S_k = sum_i |X[i,k]| accumulated
 * in fp64 in a fixed order: rows in consecutive chunks of 256, inside a chunk one row at a time in
 * increasing order, then the chunk totals in chunk order. Deterministic and bit-reproducible.
 *   X         device, bf16 [N, K], row stride ldx (elements)
 *   workspace device, >= awq_act_stats_workspace_size(N, K) bytes, contents need not be initialised
 *   act_mean  device, float [K] (output)
 * Requires N >= 1, K >= 1, K % 2 == 0 and ceil(N / 256) <= 65535 (N <= 16,776,960), else
 * AWQ_ERR_INVALID_ARG before any launch.
 * ------------------------------------------------------------------------------------------------- */
AWQ_API size_t awq_act_stats_workspace_size(int64_t N, int64_t K);
AWQ_API awq_status awq_act_stats(const void *X, int64_t N, int64_t K, int64_t ldx, void *workspace,
                         size_t ws_bytes, float *act_mean, awq_stream_t stream);

/* ---------------------------------------------------------------------------------------------------
 * Activation statistic that allocates nothing. The pages have no counterpart: this is a deployment
 * convenience. Some callers cannot call cudaMalloc when they invoke the statistic: a plugin running
 * inside an inference engine that owns all device memory and forbids allocation on its execution path,
 * or a process that reserved nearly all HBM up front (KV caches, weight pools) where cudaMalloc would
 * fail or implicitly synchronise the device. For them this variant takes no workspace: its fp64 chunk
 * sums live in a fixed 16 MiB device array inside the library (AWQ_NOALLOC_SCRATCH_DOUBLES doubles),
 * which every GPU that loads the library holds until the process exits.
 *   Same inputs, output and result as awq_act_stats (bit-identical act_mean).
 *   Limit: ceil(N / 256) * K <= AWQ_NOALLOC_SCRATCH_DOUBLES, else AWQ_ERR_INVALID_ARG and no launch
 *   (e.g. N = 16384 with K <= 32768, or N = 4096 with K <= 131072).
 *   The first call on each device looks up the array's device address (cudaGetSymbolAddress, which may
 *   load the library's device code on that device); make that first call before any stream capture.
 *   The address is kept per device and CUDA context: after cudaDeviceReset (a new primary context, in
 *   which the library's device code and the array are loaded afresh) the next call looks it up again,
 *   so that call too belongs before any capture.
 *   All calls share the one array, which keeps the last call's contents (every value a call reads is
 *   first written by that call, so nothing needs clearing): calls that overlap on the GPU, e.g. on two
 *   streams, race and give wrong results. Serialise them.
 * ------------------------------------------------------------------------------------------------- */
#define AWQ_NOALLOC_SCRATCH_DOUBLES (1ull << 21)
AWQ_API awq_status awq_act_stats_noalloc(const void *X, int64_t N, int64_t K, int64_t ldx, float *act_mean,
                                         awq_stream_t stream);

/* ---------------------------------------------------------------------------------------------------
 * (2) Scale table alone (the first stage of awq_search, exposed for testing and for callers that want
 * the candidates). Row j of table (device, float [n_grid, K]) receives, with r = RN32(j / n_grid):
 *   t = correctly rounded fp32 of act_mean[k]^r (0^0 = 1), t = max(t, RN32(1e-4)),
 *   d = RN32(sqrt(RN32(max_k t * min_k t))), s = RN32(t / d).
 * flags: 0 or AWQ_FLAG_EXACT_POW, optionally with one of the alternative rules (also accepted by
 * awq_search_ex), all bit-exact, P_j = RN32(j / (n_grid - 1)) (linspace(0, 1, n_grid), 1.0 included):
 *   AWQ_FLAG_SCALES_WEIGHT_AWARE: t = max(RN32(CR32(a^P) / RN32(CR32(wm^RN32(1 - P)) + RN32(1e-6))), 1e-4),
 *     then the same geometric normalisation; wm[k] = mean_o |W[o,k]| (fixed order as in (1)); only through
 *     awq_scale_table_ex (which takes wm) or awq_search_ex.
 *   AWQ_FLAG_SCALES_RMS: t = CR32(max(a, RN32(1e-5))^P); m = RN32(RN64(S / K)), S = fp64 sum of RN32(t^2)
 *     in 256-column chunks (in order, chunk totals in order); s = max(RN32(t / RN32(sqrt(m))), 1e-4)
 *     (n_grid = 11 gives the page's 0, 0.1, ..., 1.0).
 * 1 <= n_grid <= AWQ_MAX_N_GRID.
 * ------------------------------------------------------------------------------------------------- */
AWQ_API size_t awq_scale_table_workspace_size(int64_t K, int n_grid);
AWQ_API awq_status awq_scale_table(const float *act_mean, int64_t K, int n_grid, unsigned flags, void *workspace,
                           size_t ws_bytes, float *table, awq_stream_t stream);
AWQ_API awq_status awq_scale_table_ex(const float *act_mean, const float *weight_mean, int64_t K, int n_grid,
                                      unsigned flags, void *workspace, size_t ws_bytes, float *table,
                                      awq_stream_t stream);

/* ---------------------------------------------------------------------------------------------------
 * (2)-(4) The search. For every candidate j it forms the weight error dW_j = W - W_hat_j (fp32, rounded
 * to bf16) and evaluates loss_j = sum((X dW_j^T)^2) / (N * O) with tensor cores (bf16 x bf16, fp32
 * accumulation in tensor memory, squares reduced in fp32 per row and fp64 across rows and tiles in a
 * fixed order); the [N, O] product is never written to memory.
 *   X, W       device bf16 as above; W holds the stacked rows of every linear that reads X
 *   act_mean   device float [K] (from awq_act_stats or the caller)
 *   workspace  device, >= awq_search_workspace_size(N, K, O, group, n_grid) bytes, 1024-byte aligned
 *   losses     device double [n_grid] (output)
 *   best_j     device int (output): first index of the minimum loss; -1 after a device timeout
 *   scales     device float [K] (output): row best_j of the scale table
 * The scales, and the codes/steps/zeros that awq_quantize_pack derives from them, are bit-exact
 * functions of (act_mean, W); the losses carry bf16 rounding of dW and fp32 tensor-core accumulation.
 * Requires N >= 1, O >= 1, K >= 128, K % 128 == 0, N, O, K < 2^31, 1 <= n_grid <= AWQ_MAX_N_GRID.
 * group: 128 (INT4 groups of 128 in-features), or 0 (per output channel) together with
 * AWQ_FLAG_QUANT_INT8; the workspace size is the same for both.
 * ------------------------------------------------------------------------------------------------- */
AWQ_API size_t awq_search_workspace_size(int64_t N, int64_t K, int64_t O, int group, int n_grid);
AWQ_API awq_status awq_search(const void *X, int64_t N, int64_t K, int64_t ldx, const void *W, int64_t O,
                      int64_t ldw, const float *act_mean, int group, int n_grid, void *workspace,
                      size_t ws_bytes, double *losses, int *best_j, float *scales, awq_stream_t stream);
/* Same, with flags (AWQ_FLAG_EXACT_DIVISION, AWQ_FLAG_EXACT_POW, AWQ_FLAG_INJECT_STALL, one of
 * AWQ_FLAG_SCALES_WEIGHT_AWARE / AWQ_FLAG_SCALES_RMS to search the alternative candidate scales, and
 * AWQ_FLAG_QUANT_INT8 with group 0 to search with the INT8 per-channel quantizer of (5b)). */
AWQ_API awq_status awq_search_ex(const void *X, int64_t N, int64_t K, int64_t ldx, const void *W, int64_t O,
                         int64_t ldw, const float *act_mean, int group, int n_grid, unsigned flags,
                         void *workspace, size_t ws_bytes, double *losses, int *best_j, float *scales,
                         awq_stream_t stream);

/* Synchronises `stream`, then reads the device status word of a workspace last used by awq_search:
 * AWQ_OK or AWQ_ERR_TIMEOUT (message names the wait that gave up). */
AWQ_API awq_status awq_search_status(const void *workspace, size_t ws_bytes, awq_stream_t stream);

/* Where awq_search leaves its per-tile partial sums inside the workspace (valid after the call):
 * double partial[n_grid][tiles_o][tiles_n][partials_per_tile] at byte offset partials_offset;
 * partial[j][a][b][e] is the sum of squares of the outputs of token rows
 * [b*tile_n + e*r, b*tile_n + (e+1)*r), r = tile_n / partials_per_tile, and output rows
 * [a*tile_o, (a+1)*tile_o) for candidate j (rows past N or O contribute zero). */
typedef struct awq_search_layout {
  int64_t tile_n, tile_o;   /* tile extent along tokens and along output rows */
  int64_t tiles_n, tiles_o; /* tiles per candidate along tokens and along output rows */
  int64_t partials_per_tile;
  size_t partials_offset;   /* bytes from the workspace start */
  size_t workspace_bytes;   /* same as awq_search_workspace_size() */
} awq_search_layout;
AWQ_API awq_status awq_search_get_layout(int64_t N, int64_t K, int64_t O, int group, int n_grid,
                                 awq_search_layout *out /* host */);

/* Measurement hook: when set (non-NULL), every later awq_search* call on this thread records the CUDA
 * event `before` on its stream right before the loss-GEMM launch and `after` right after it, so a caller
 * can time that kernel alone. Both are cudaEvent_t handles created by the caller; pass NULL, NULL to
 * stop. */
AWQ_API void awq_set_profile_events(void *before_loss_gemm, void *after_loss_gemm);

/* ---------------------------------------------------------------------------------------------------
 * (5) Codes of W at given scales (normally the `scales` output of awq_search):
 *   codes  device uint32 [O, K/8]: code of in-feature k at bits 4*(k%8) of word k/8
 *   steps  device float [O, K/group]: per-group step
 *   zeros  device float [O, K/group]: per-group zero point (integer-valued, not clamped, never -0)
 * Bit-exact: every operation is one IEEE fp32 operation in the order given in (3).
 * ------------------------------------------------------------------------------------------------- */
AWQ_API awq_status awq_quantize_pack(const void *W, int64_t O, int64_t K, int64_t ldw, const float *scales,
                             int group, uint32_t *codes, float *steps, float *zeros, awq_stream_t stream);
/* Same, with flags (AWQ_FLAG_EXACT_DIVISION). */
AWQ_API awq_status awq_quantize_pack_ex(const void *W, int64_t O, int64_t K, int64_t ldw, const float *scales,
                                int group, unsigned flags, uint32_t *codes, float *steps, float *zeros,
                                awq_stream_t stream);

/* ---------------------------------------------------------------------------------------------------
 * (5b) Symmetric INT8 codes of W at given scales, one step per output channel (formula of section 2.1
 * of the hncyxsy.com large-model outlier article, with the per-channel weight setting of the
 * quantization YAML on the msModelSlim page). With w' = RN32(w * s_k) over the row's K in-features:
 *   step_o = max(RN32(max_k |w'| / 127), RN32(1e-5))    q = min(max(rint(RN32(w' / step_o)), -127), 127)
 * and the dequantized value is RN32(q * step_o). The search with AWQ_FLAG_QUANT_INT8 scores exactly this
 * quantizer (w_hat = RN32(q * step_o) * RN32(1 / s_k), as for INT4).
 *   W      device bf16 [O, ldw] as in awq_search
 *   scales device float [K], 16-byte aligned
 *   codes  device int8 [O, K] row-major (row stride K), 8-byte aligned (output)
 *   steps  device float [O] (output)
 *   flags  0 or AWQ_FLAG_EXACT_DIVISION
 * Bit-exact: every operation is one IEEE fp32 operation in the order above. Requires K % 8 == 0.
 * ------------------------------------------------------------------------------------------------- */
AWQ_API awq_status awq_quantize_pack_int8(const void *W, int64_t O, int64_t K, int64_t ldw, const float *scales,
                                          unsigned flags, int8_t *codes, float *steps, awq_stream_t stream);

/* ---------------------------------------------------------------------------------------------------
 * Applying the chosen scales (SubgraphFusionFactory step of 缩放因子搜索流程 on the msModelSlim page):
 * the target linears get forward scaling of their input columns, W' = W diag(s); the producer of their
 * input gets the inverse: the norm weight gamma' = gamma / s (NormLinearSubgraph), or the output rows
 * (and bias) of the source linear divided by s (LinearLinearSubgraph linear1, OVSubgraph v_proj for
 * multi-head attention, UpDownSubgraph up_proj), so that section 一's identity
 * X W^T = (X diag(s)^-1)(diag(s) W)^T keeps the subgraph's output.
 *   awq_scale_columns: out[r, c] = bf16(RN32(A[r, c] op s[c]))
 *   awq_scale_rows:    out[r, c] = bf16(RN32(A[r, c] op s[r]))
 * op = AWQ_SCALE_MULTIPLY or AWQ_SCALE_DIVIDE (IEEE fp32 division); A, out bf16 row-major with row
 * strides lda, ldo (multiples of 8); C % 8 == 0; out may equal A (in place). A norm weight or a bias is
 * a 1 x C matrix. Bit-exact.
 * ------------------------------------------------------------------------------------------------- */
#define AWQ_SCALE_MULTIPLY 0
#define AWQ_SCALE_DIVIDE 1
AWQ_API awq_status awq_scale_columns(const void *A, int64_t R, int64_t C, int64_t lda, const float *s, int op,
                                     void *out, int64_t ldo, awq_stream_t stream);
AWQ_API awq_status awq_scale_rows(const void *A, int64_t R, int64_t C, int64_t lda, const float *s, int op,
                                  void *out, int64_t ldo, awq_stream_t stream);

/* ---------------------------------------------------------------------------------------------------
 * Deployment GEMM of a quantized linear (W4A16): Y = X' deq(W)^T, the weights read as the packed codes,
 * steps and zeros of awq_quantize_pack and dequantized on the fly ("GPU 硬件级反量化算子内联融合" on the
 * bjdmk.com.cn AWQ article), deq(W)[o, k] = (q[o,k] - z[o,g]) * step[o,g], g = k / 128.
 * X' is the layer input with the AWQ scales already folded out (X diag(s)^-1, e.g. by awq_scale_columns
 * on the previous norm weight). fp32 accumulation on the tensor cores, bf16 output. The weight enters as:
 *   M > 64 tokens:  bf16(RN32(RN32(q - z) * step)), dequantized into the tensor-core operand tiles;
 *   M <= 64 tokens: its exact value: the tensor cores sum (128 + q) * x' per group of 128 in-features
 *                   (exact bf16 operands) and the step and zero point are applied per group and output,
 *                   Y = sum_g step_g * (S_g - (128 + z_g) * sum_{k in g} x'_k), in fp32.
 *   X       device bf16 [M, K], row stride ldx (multiple of 8)
 *   codes   device uint32 [O, K/8], steps / zeros device float [O, K/128] (contiguous, as packed)
 *   Y       device bf16 [M, O], row stride ldy (multiple of 8)
 *   workspace  device, >= awq_w4a16_workspace_size(K, O) bytes, ZERO-FILLED BEFORE ITS FIRST USE
 *              (e.g. cudaMemsetAsync once after allocating it). It holds the status word and a tile
 *              counter, a fixed 256 KB region of per-block counters (M <= 64 tokens; every call leaves
 *              them at zero, and nothing else writes there, so one zero fill serves all later calls
 *              whatever their shapes), a group-major copy of steps and zeros (many tokens), and for
 *              M <= 64 a permuted copy of X (64 rows), its per-group sums and split-K partial sums.
 *              After a device timeout the counters may be left set: zero-fill the workspace again
 *              before reusing it. M <= 64 is two launches on `stream`: a small kernel that writes the
 *              X copy and group sums, and the GEMM as its programmatic dependent (it starts early and
 *              waits for them).
 * Requires K % 128 == 0, O % 8 == 0, M >= 1. M <= 64 runs a few-token kernel (weight rows on the MMA's M
 * side, groups split across CTAs, partial sums added in a fixed order). Both are deterministic. A device
 * timeout is reported by awq_search_status() on the same workspace.
 * ------------------------------------------------------------------------------------------------- */
AWQ_API size_t awq_w4a16_workspace_size(int64_t K, int64_t O);
AWQ_API awq_status awq_w4a16_gemm(const void *X, int64_t M, int64_t K, int64_t ldx, const uint32_t *codes,
                                  const float *steps, const float *zeros, int64_t O, void *Y, int64_t ldy,
                                  void *workspace, size_t ws_bytes, awq_stream_t stream);

/* ---------------------------------------------------------------------------------------------------
 * One-token products (W4A16): the deployment GEMM's form for the 1 to 8 tokens of a decode step, in one
 * launch and without a workspace. Weights, X' and the value of a weight as in awq_w4a16_gemm for few tokens
 * (the weight enters with its exact value, fp32 sums, one rounding to bf16 at the end).
 *   gated = 0: Y[m, o] = sum_k X'[m, k] deq(W)[o, k] (+ bias[o]);  Y is [M, O]
 *   gated = 1: the rows of W are a gate projection's O/2 rows, then an up projection's O/2 rows;
 *              Y[m, i] = a / (1 + exp(-a)) * b in fp32, a = row i's product, b = row O/2 + i's; Y is [M, O/2]
 *   X       device bf16 [M, K], row stride ldx (multiple of 8), 16-byte aligned
 *   codes   device uint32 [O, K/8], 16-byte aligned; steps / zeros device float [O, K/128] (as packed)
 *   bias    device bf16 [O] or NULL (NULL when gated)
 *   Y       device bf16, row stride ldy >= its columns (no alignment beyond 2 bytes); must not overlap X
 * Requires 1 <= M <= AWQ_GEMV_MAX_TOKENS, K % 128 == 0, any O >= 1 (gated: even; at most 8388480 rows, half
 * of that per projection when gated). Deterministic. An infinity or a NaN in a row of X makes of that row's outputs what the
 * formula makes of it, and of no other's (so in awq_w4a16_experts too).
 * ------------------------------------------------------------------------------------------------- */
#define AWQ_GEMV_MAX_TOKENS 8
AWQ_API awq_status awq_w4a16_gemv(const void *X, int64_t M, int64_t K, int64_t ldx, const uint32_t *codes,
                                  const float *steps, const float *zeros, int64_t O, const void *bias, int gated,
                                  void *Y, int64_t ldy, awq_stream_t stream);

/* ---------------------------------------------------------------------------------------------------
 * Tokens sorted by expert. Slot s = t * top_k + j is the j-th pick of token t; ids holds the expert of every
 * slot (int32 or int64, id_bytes 4 or 8). An id outside [0, E) names no expert (a padded token, an expert of
 * another device): its slot has no row.
 *   offsets  device int32 [E + 1]: first sorted row of each expert; offsets[E] = number of routed slots
 *   order    device int32 [n_slots]: slot of each sorted row, rows in order of (expert, slot); -1 from
 *            offsets[E] on
 *   pos      device int32 [n_slots]: sorted row of each slot, -1 where there is none
 *   workspace  device, >= awq_expert_sort_workspace_size(n_slots, E) bytes (0 for up to 4096 slots: may be
 *            NULL then), contents need not be initialised
 * Requires 1 <= n_slots < 2^31, 1 <= E <= AWQ_MAX_EXPERTS. A token may pick the same expert twice. Stable and
 * deterministic.
 * ------------------------------------------------------------------------------------------------- */
#define AWQ_MAX_EXPERTS 1024
AWQ_API size_t awq_expert_sort_workspace_size(int64_t n_slots, int64_t E);
AWQ_API awq_status awq_expert_sort(const void *ids, int id_bytes, int64_t n_slots, int64_t E, void *workspace,
                                   size_t ws_bytes, int32_t *offsets, int32_t *order, int32_t *pos,
                                   awq_stream_t stream);

/* Rows in expert order and back. T tokens, top_k picks each; Xs, Ys, dXs, dYs are bf16 [T * top_k, columns] in
 * sorted rows; matrices as everywhere (16-byte aligned, row strides and columns multiples of 8); offsets,
 * order and pos from awq_expert_sort. Sums are fp32 in slot order, rounded once to bf16. Rows from offsets[E] on are
 * neither read nor written. No input may overlap an output.
 *   awq_expert_gather:           Xs[r] = X[order[r] / top_k]; with scales (device float [E, K], 16-byte aligned)
 *                                bf16(RN32(X / scales[e])), e the row's expert (the same bits as
 *                                awq_scale_columns with AWQ_SCALE_DIVIDE)
 *   awq_expert_gather_backward:  its gradient dX[t] = sum_j RN32(dXs[pos[t, j]] / scales[e]) (scales as there)
 *   awq_expert_combine:          Y[t] = sum_j weights[t, j] * Ys[pos[t, j]] (weights device float [T, top_k], or
 *                                NULL for ones); 0 for a token without a row
 *   awq_expert_combine_backward: its gradients dYs[pos[t, j]] = weights[t, j] * dY[t] (bf16) and
 *                                dweights[t, j] = <dY[t], Ys[pos[t, j]]> (device float [T, top_k], fp32 sum in a
 *                                fixed order; 0 where a slot has no row) */
AWQ_API awq_status awq_expert_gather(const void *X, int64_t T, int64_t K, int64_t ldx, int64_t top_k,
                                     const int32_t *offsets, int64_t E, const int32_t *order, const float *scales,
                                     void *Xs, int64_t ldxs, awq_stream_t stream);
AWQ_API awq_status awq_expert_gather_backward(const void *dXs, int64_t T, int64_t K, int64_t lddxs, int64_t top_k,
                                              const int32_t *offsets, int64_t E, const int32_t *pos,
                                              const float *scales, void *dX, int64_t lddx, awq_stream_t stream);
AWQ_API awq_status awq_expert_combine(const void *Ys, int64_t T, int64_t O, int64_t ldys, int64_t top_k,
                                      const int32_t *pos, const float *weights, void *Y, int64_t ldy,
                                      awq_stream_t stream);
AWQ_API awq_status awq_expert_combine_backward(const void *dY, int64_t T, int64_t O, int64_t lddy, const void *Ys,
                                               int64_t ldys, int64_t top_k, const int32_t *pos, const float *weights,
                                               void *dYs, int64_t lddys, float *dweights, awq_stream_t stream);

/* ---------------------------------------------------------------------------------------------------
 * Products of the experts (W4A16): Y[r] = Xs[r] deq(W_e)^T for the rows offsets[e] <= r < offsets[e + 1] of
 * every expert e, or with gated = 1 the gated form of awq_w4a16_gemv. The weights enter with
 * their exact value, (q - z) summed per group and scaled by the fp32 step; only in a group with |z| > 240 (its
 * weights nearly equal) an expert with more than 8 rows takes q - z rounded to bf16. zeros must be whole numbers, as packing
 * gives them: with more than 8 rows another z enters rounded to bf16.
 *   Xs      device bf16 [R, K] sorted rows, row stride ldx (multiple of 8)
 *   codes   device uint32 [E, O, K/8], 16-byte aligned; steps / zeros device float [E, O, K/128] (as packed:
 *           integer-valued zeros)
 *   Y       device bf16 [R, O] (gated: [R, O/2]), row stride ldy >= its columns; rows from offsets[E] on are left
 *           as they were; must not overlap Xs
 *   workspace  device, 16-byte aligned, >= awq_w4a16_experts_workspace_size(R, E, K, O) bytes, ZERO-FILLED
 *           BEFORE ITS FIRST USE and after a device timeout, which awq_search_status() reports on it: rows of
 *           experts with more than 8 rows may then be left as they were, in that call and until it is zeroed
 * Requires K % 128 == 0, any O >= 1 (gated: even), 1 <= E <= AWQ_MAX_EXPERTS. Deterministic.
 * ------------------------------------------------------------------------------------------------- */
AWQ_API size_t awq_w4a16_experts_workspace_size(int64_t R, int64_t E, int64_t K, int64_t O);
AWQ_API awq_status awq_w4a16_experts(const void *Xs, int64_t R, int64_t K, int64_t ldx, const int32_t *offsets,
                                     int64_t E, const uint32_t *codes, const float *steps, const float *zeros,
                                     int64_t O, int gated, void *Y, int64_t ldy, void *workspace, size_t ws_bytes,
                                     awq_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* AWQ_B200_H */
